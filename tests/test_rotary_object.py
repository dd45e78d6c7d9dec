"""What a Rotary holds, without a GPU."""
import copy
import math
import pickle

import numpy as np
import pytest

from ragged_blocked_kv_gb300.layer import DecoderLayer
from test_draft_host import _append, _rotary
from test_step_host import INVALID

OTHERS = {"rotary_dim": 32, "layout": "interleaved", "scale": 2.0,
          "inv_freq": np.ones(32), "turns": None}


@pytest.mark.parametrize("name", OTHERS)
def test_what_calls_hold_cannot_be_replaced(rbkv, name):
    """Calls hold the table's address, and the values as they were: a replaced table would be
    read after it was freed, a replaced value not at all."""
    r = rbkv.Rotary(64, device="cpu")
    before, held = getattr(r, name), r._c._obj.turns
    with pytest.raises(AttributeError, match="make another Rotary"):
        setattr(r, name, before.clone() if name == "turns" else OTHERS[name])
    with pytest.raises(AttributeError, match="cannot be deleted"):
        delattr(r, name)
    assert getattr(r, name) is before and held == r.turns.data_ptr()
    setattr(r, name, before)                             # (itself: nothing changes)


def test_angles_are_the_objects_own(rbkv):
    """The table is made from a copy of what is given, and the copy does not change."""
    given = np.array([1.0, 0.5])
    r = rbkv.Rotary(4, inv_freq=given, device="cpu")
    given[0] = 3.0
    assert r.inv_freq.tolist() == [1.0, 0.5]
    for x in (r, rbkv.Rotary(4, device="cpu")):
        with pytest.raises(ValueError):
            x.inv_freq[0] = 2.0


@pytest.mark.parametrize("scale", [math.nan, math.inf, -math.inf, 1e39, -1e300])
def test_scales_that_are_not_finite_are_refused(rbkv, scale):
    """(in fp32, the type that calls take)"""
    with pytest.raises(ValueError, match="scale must be finite"):
        rbkv.Rotary(64, scale=scale, device="cpu")
    assert _append(rbkv, r=_rotary(rbkv, scale=scale)) == INVALID
    assert b"scale" in rbkv.lib().rbkv_last_error()


def test_scales_that_are_finite(rbkv):
    for scale in (0.0, -1.5, 3e38, 1e-45):
        assert rbkv.Rotary(64, scale=scale, device="cpu").scale == scale


@pytest.mark.parametrize("how", [copy.copy, copy.deepcopy, lambda x: pickle.loads(pickle.dumps(x))],
                         ids=["copy", "deepcopy", "pickle"])
def test_copies_hold_their_own_table(rbkv, how):
    r = rbkv.Rotary(64, layout="interleaved", scale=1.5, device="cpu")
    s = how(r)
    want = (r.turns.tolist(), r.inv_freq.tolist(), 64, "interleaved", 1.5)
    mine = s.turns.data_ptr()
    assert (mine == r.turns.data_ptr()) == (how is copy.copy)
    del r
    assert (s.turns.tolist(), s.inv_freq.tolist(), s.rotary_dim, s.layout, s.scale) == want
    c = s._c._obj
    assert (c.turns, c.rotary_dim, c.interleaved, c.scale) == (mine, 64, 1, 1.5)
    with pytest.raises(AttributeError, match="make another Rotary"):
        s.turns = s.turns.clone()
    with pytest.raises(ValueError):
        s.inv_freq[0] = 2.0


def test_a_layer_with_rotary_positions_can_be_copied(rbkv):
    layer = DecoderLayer(None, {}, 2, 1, 64, rotary=rbkv.Rotary(64, device="cpu"))
    other = copy.deepcopy(layer)
    assert other.rotary.turns.tolist() == layer.rotary.turns.tolist()
    assert other.rotary._c._obj.turns == other.rotary.turns.data_ptr()
