"""Block ids outside the pool in a step's tables or prefix list: the keys they
stand for are left out of the softmax, on every route, and reported."""
import math

import numpy as np
import pytest
import torch

from step_harness import error_bound, i32
from test_gpu_step import BOUNDS, POKED, _case

pytestmark = pytest.mark.gpu

BAD = (-2, -1, 10 ** 6, -2 ** 31)


def _without(want, q, kc, vc, table, ids, prefix):
    """`step_harness.reference` over the keys whose block is in the pool, row by
    row; a row without one is 0."""
    T, (H_q, D) = int(want.q_start[-1]), q.shape[1:]
    N, H_kv, B = kc.shape[:3]
    out = torch.zeros(T, H_q, D, dtype=torch.float64)
    absv, absqk = torch.zeros_like(out), torch.zeros(T, H_q, 1, dtype=torch.float64)
    keys = torch.zeros(T, 1, 1, dtype=torch.float64)
    seq = np.searchsorted(want.q_start[1:], np.arange(T), side="right")
    for r in range(T):
        places = [(int(ids[p // B]), p % B) for p in range(prefix)]
        places += [(int(table[seq[r], p // B]), p % B) for p in range(int(want.position[r]) + 1)]
        places = np.array([x for x in places if 0 <= x[0] < N]).reshape(-1, 2)
        if len(places) == 0:
            continue
        b, off = torch.from_numpy(places).T
        k, v = (c[b, :, off].double().repeat_interleave(H_q // H_kv, 1).transpose(0, 1)
                for c in (kc, vc))                                  # [H_q, keys, D]
        qr = q[r].double()[:, None]
        w = torch.softmax(qr @ k.transpose(1, 2) / math.sqrt(D), -1)
        out[r], absv[r] = (w @ v)[:, 0], (w @ v.abs())[:, 0]
        absqk[r] = (qr.abs() @ k.abs().transpose(1, 2) / math.sqrt(D)).amax(-1)
        keys[r] = len(places)
    return out, absv, absqk, keys


def _poke(rbkv, shape, seen, n_new, prefix, bad_prefix, bad_own, value, seed=0):
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, prefix, seen, n_new, pad=3,
                                                  seed=seed)
    ids, table = np.array(ids), want.table.copy()
    for i in bad_prefix:
        ids[i] = value
    for s, c in bad_own:
        assert c < -(-want.ctx[s] // shape[3])
        table[s, c] = value
    t.block_table.copy_(i32(table))
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    t.attention(q.cuda(), kd, vd, prefix_table=i32(ids) if prefix else None, prefix_len=prefix,
                o=o)
    with pytest.raises(rbkv.RbkvError) as e:
        t.device_status()
    assert e.value.status == BOUNDS
    ref = _without(want, q, kc, vc, table, ids, prefix)
    err = (o[:rows].cpu().double() - ref[0]).abs()
    assert (err <= error_bound(ref, shape[2], shape[4])).all(), float(err.max())
    assert (o[rows:] == 7.0).all()


SHAPES = [(32, 8, 128, 64, "bf16"), (8, 4, 128, 8, "bf16"), (16, 1, 128, 128, "bf16"),
          (7, 1, 128, 256, "bf16"), (8, 8, 128, 16, "bf16"), (8, 2, 64, 16, "bf16"),
          (8, 2, 32, 5, "f32")]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("value", BAD)
def test_bad_prefix_ids_are_left_out(rbkv, shape, value):
    """Whole key tiles and parts of one, the list's first and last entry."""
    B = shape[3]
    n = -(-700 // B)
    _poke(rbkv, shape, *POKED, 700, sorted({0, n // 2, n - 1} if n < 9 else
                                           {0, 3, 4, n // 2, n - 1}), [], value)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("prefix", [0, 130])
@pytest.mark.parametrize("value", BAD)
def test_bad_own_ids_are_left_out(rbkv, shape, prefix, value):
    """Ids of cached and of new tokens, in a long chunk, a short one and single
    tokens; one row whose every own key is gone."""
    B = shape[3]
    own = [(0, 0), (0, 369 // B), (3, 150 // B), (4, 500 // B), (4, 1015 // B), (5, 0)]
    _poke(rbkv, shape, *POKED, prefix, [], own + ([(5, 1)] if B <= 8 else []), value, seed=1)


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (16, 16, 128, 8, "bf16"),
                                   (8, 2, 64, 16, "f32")], ids=str)
@pytest.mark.parametrize("value", BAD)
def test_bad_ids_in_steps_of_few_rows(rbkv, shape, value):
    """One row: the prefix, too, is streamed.  Then nothing but bad ids."""
    B = shape[3]
    _poke(rbkv, shape, [300], [1], 500, [0, 400 // B, 499 // B], [(0, 100 // B)], value)
    blocks = range(-(-301 // B))
    _poke(rbkv, shape, [300], [1], 500, range(-(-500 // B)), [(0, c) for c in blocks], value)
    _poke(rbkv, shape, [300], [1], 0, [], [(0, c) for c in blocks], value)
