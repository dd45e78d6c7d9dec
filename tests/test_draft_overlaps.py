"""Caches that lie on the arrays of a step, without a GPU: refused before anything is
launched."""
import ctypes as C

import pytest

from test_draft_host import FAR, _append, _draft
from test_step_host import INVALID, _cfg, _tables

# (32 blocks of 16 rows of 2 heads of 64 in fp32: 256 KB a cache)
AT = 20 * FAR
TABLES = ("q_start", "position", "slot", "plan", "status")
DRAFT = ("place", "path", "accepted", "work")


def _with(rbkv, name, at):
    """Tables and a draft of which `name` lies at `at`."""
    t = _tables(rbkv, **{n: 30 * FAR + i * 4096 for i, n in enumerate(TABLES)})
    d = _draft(rbkv)
    setattr(t if name in TABLES else d, name, at)
    return t, d


@pytest.mark.parametrize("name", TABLES + DRAFT)
@pytest.mark.parametrize("end", [0, 262144 - 16])
def test_caches_on_arrays_of_the_step(rbkv, name, end):
    L, cfg = rbkv.lib(), _cfg(rbkv)
    t, d = _with(rbkv, name, AT + end)
    for k, v in ((AT, 40 * FAR), (40 * FAR, AT)):
        assert _append(rbkv, t=t, d=d, kc=k, vc=v) == INVALID
        assert b"array of the step" in L.rbkv_last_error()
        assert L.rbkv_step_draft_compact(C.byref(cfg), C.byref(t), C.byref(d), k, v,
                                         None) == INVALID
        assert b"array of the step" in L.rbkv_last_error()
        if name in TABLES:
            assert _append(rbkv, t=t, kc=k, vc=v) == INVALID
            assert b"array of the step" in L.rbkv_last_error()
    assert _append(rbkv, t=t, d=d, q_out=AT + end) == INVALID
