"""Drafted tokens and rotary positions without a GPU: refusals of the C entries
(before anything is launched), the binding's checks, the oracle's own pins."""
import ctypes as C
import math

import numpy as np
import pytest
import torch

import oracle
from draft_harness import draft_reference, random_trees
from step_harness import random_batch, reference
from test_step_host import FAKE, INVALID, UNSUPPORTED, _cfg, _tables

D = oracle.draft
FAR = 1 << 32            # (fake addresses far enough apart not to overlap)


def _draft(rbkv, **change):
    d = rbkv._StepDraft(*(FAR + (i << 20) for i in range(6)))
    for k, v in change.items():
        setattr(d, k, v)
    return d


def _rotary(rbkv, **change):
    r = rbkv._Rotary(2 * FAR, 64, 0, 1.0)
    for k, v in change.items():
        setattr(r, k, v)
    return r


def _append(rbkv, cfg=None, t=None, d=None, r=None, prefix=0, q=3 * FAR, q_out=3 * FAR, k=4 * FAR,
            v=5 * FAR, kc=6 * FAR, vc=7 * FAR):
    cfg, t = cfg or _cfg(rbkv), t or _tables(rbkv)
    return rbkv.lib().rbkv_step_append_rotary(
        C.byref(cfg), C.byref(t), None if d is None else C.byref(d),
        C.byref(_rotary(rbkv) if r is None else r), prefix, q, q_out, k, v, kc, vc, None)


def test_rotary_refusals(rbkv):
    for change in ({"turns": None}, {"turns": 2 * FAR + 4}, {"rotary_dim": 0}, {"rotary_dim": 66},
                   {"rotary_dim": 7}, {"rotary_dim": -2}, {"interleaved": 2}, {"interleaved": -1}):
        assert _append(rbkv, r=_rotary(rbkv, **change)) == INVALID, change
    for name in ("q", "q_out", "k", "v", "kc", "vc"):
        assert _append(rbkv, **{name: None}) == INVALID, name
        assert _append(rbkv, **{name: 8 * FAR + 8}) == INVALID, name
    # q_out on part of q, on the new rows, on the caches, on what the call reads
    for at in (3 * FAR + 16, 4 * FAR, 5 * FAR, 6 * FAR + 1024, 7 * FAR, 2 * FAR, FAKE):
        assert _append(rbkv, q_out=at) == INVALID, hex(at)
    assert _append(rbkv, kc=6 * FAR, vc=6 * FAR) == INVALID          # one cache for both
    assert _append(rbkv, kc=6 * FAR, vc=6 * FAR + 65536) == INVALID  # (32 blocks of 8 KB)
    for name in ("q", "k", "v"):
        assert _append(rbkv, **{"q_out": 9 * FAR, name: 7 * FAR + 64}) == INVALID, name
    assert _append(rbkv, prefix=-1) == INVALID and _append(rbkv, prefix=(1 << 30) + 1) == INVALID
    assert _append(rbkv, d=_draft(rbkv, place=None)) == INVALID
    assert _append(rbkv, d=_draft(rbkv, place=9 * FAR), q_out=9 * FAR) == INVALID
    assert _append(rbkv, cfg=_cfg(rbkv, 1 << 18, 1 << 18, 64)) == UNSUPPORTED
    assert _append(rbkv, t=_tables(rbkv, max_tokens=0)) == INVALID
    L = rbkv.lib()
    r = C.byref(_rotary(rbkv))
    args = [3 * FAR, 3 * FAR, 4 * FAR, 5 * FAR, 6 * FAR, 7 * FAR, None]
    assert L.rbkv_kv_append_rotary(None, r, *args) == INVALID
    assert L.rbkv_frame_kv_append_rotary(None, r, *args) == INVALID
    comp = rbkv.Composer(rbkv.Config(8, 2, 64, 16, "f32", 10))
    p = comp.compose(20, 0, [(1, 20, 0)])
    for i in range(6):
        assert L.rbkv_kv_append_rotary(p._h, r, *args[:i], None, *args[i + 1:]) == INVALID
    assert L.rbkv_kv_append_rotary(p._h, None, *args) == INVALID
    assert L.rbkv_kv_append_rotary(p._h, C.byref(_rotary(rbkv, rotary_dim=128)), *args) == INVALID
    assert comp.compose(0, 0, []).num_tokens == 0


def test_draft_refusals(rbkv):
    L, cfg, t = rbkv.lib(), _cfg(rbkv), _tables(rbkv)

    def calls(d, t=t):
        c, t = C.byref(cfg), C.byref(t)
        d = None if d is None else C.byref(d)
        a = 9 * FAR
        return [L.rbkv_step_draft_plan(c, t, d, a, None),
                L.rbkv_step_draft_accept(c, t, d, a, a, None, None),
                L.rbkv_step_draft_compact(c, t, d, a, 10 * FAR, None),
                L.rbkv_step_attention_draft(c, t, d, a, a, a, None, 0, 10 * FAR, 11 * FAR, 1 << 30,
                                            None)]

    for bad in (None, *(_draft(rbkv, **x) for x in (
            {"place": None}, {"ancestors": None}, {"path": None}, {"accepted": None},
            {"next_token": None}, {"work": None}, {"work": FAR + 8}, {"ancestors": FAR + 4}, {"place": FAR + 2}, {"path": FAR + 1},
            {"accepted": FAR + 2}, {"next_token": FAR + 3}))):
        assert calls(bad) == [INVALID] * 4
    assert calls(_draft(rbkv), _tables(rbkv, num_seqs=0)) == [INVALID] * 4
    c, tt, d = C.byref(cfg), C.byref(t), C.byref(_draft(rbkv))
    a, place = 9 * FAR, FAR
    assert L.rbkv_step_draft_plan(c, tt, d, None, None) == INVALID
    assert L.rbkv_step_draft_plan(c, tt, d, a + 2, None) == INVALID
    for at in (place, place + (1 << 20), place + (2 << 20), place + (4 << 20) + 8,
               place + (5 << 20) + 16, FAKE):
        assert L.rbkv_step_draft_plan(c, tt, d, at, None) == INVALID, hex(at)
        assert L.rbkv_step_draft_accept(c, tt, d, at, a, None, None) == INVALID
        assert L.rbkv_step_draft_accept(c, tt, d, a, at, None, None) == INVALID
        assert L.rbkv_step_draft_accept(c, tt, d, a, a, at, None) == INVALID
    assert L.rbkv_step_draft_accept(c, tt, d, None, a, None, None) == INVALID
    assert L.rbkv_step_draft_accept(c, tt, d, a, None, None, None) == INVALID
    assert L.rbkv_step_draft_accept(c, tt, d, a, a, a + 1, None) == INVALID
    assert L.rbkv_step_draft_compact(c, tt, d, None, a, None) == INVALID
    assert L.rbkv_step_draft_compact(c, tt, d, a, None, None) == INVALID
    assert L.rbkv_step_draft_compact(c, tt, d, a + 8, a, None) == INVALID
    assert L.rbkv_step_draft_compact(c, tt, d, a, a, None) == INVALID
    assert L.rbkv_step_draft_compact(c, tt, d, a, a + 65536, None) == INVALID
    attend = L.rbkv_step_attention_draft
    assert attend(c, tt, d, a, a, a, None, 0, place, None, 0, None) == INVALID    # o on place
    assert attend(c, tt, d, a, a, a, None, 3, a + 4096, None, 0, None) == INVALID


def test_rotary_tables(rbkv):
    """Turns per position in units of 2^-64, and the scalings' angles."""
    def turns(r):
        return [int(x) % 2 ** 64 for x in r.turns.tolist()]

    r = rbkv.Rotary(8, base=10000.0, device="cpu")
    theta = [1.0, 0.1, 0.01, 0.001]
    assert np.allclose(r.inv_freq, theta, rtol=1e-15)
    for got, x in zip(turns(r), theta):
        assert abs(got / 2 ** 64 - x / (2 * math.pi)) <= 2.0 ** -52 * x
    half = rbkv.Rotary(8, scaling="linear", factor=2.0, device="cpu")
    assert np.allclose(half.inv_freq, np.array(theta) / 2, rtol=1e-15)
    up = rbkv.Rotary(8, scaling="base", factor=3.0, device="cpu")
    wide = 10000.0 * 3.0 ** (8 / 6)
    assert np.allclose(up.inv_freq, [wide ** (-i / 4) for i in range(4)], rtol=1e-14)
    # 1000 positions turn the pairs 159, 15.9, 1.59 and 0.159 times
    parts = rbkv.Rotary(8, scaling="parts", factor=4.0, original_length=1000, low=1.0, high=32.0,
                        device="cpu")
    keep = [1.0, (1000 * 0.1 / (2 * math.pi) - 1) / 31, (1000 * 0.01 / (2 * math.pi) - 1) / 31, 0.0]
    assert np.allclose(parts.inv_freq, [x * (k + (1 - k) / 4) for x, k in zip(theta, keep)],
                       rtol=1e-14)
    own = rbkv.Rotary(4, inv_freq=[-0.5, 20.0], layout="interleaved", device="cpu")
    assert turns(own)[0] == 2 ** 64 - round(math.ldexp(0.5 / (2 * math.pi), 64))
    assert abs(turns(own)[1] / 2 ** 64 - (20 / (2 * math.pi)) % 1) < 1e-14
    assert rbkv.Rotary(2, scaling="base", factor=2.0, device="cpu").inv_freq.tolist() == [1.0]


@pytest.mark.parametrize("args", [
    {"rotary_dim": 0}, {"rotary_dim": 7}, {"rotary_dim": 258}, {"layout": "split"},
    {"base": 0.0}, {"base": -3.0}, {"factor": 0.0}, {"base": math.inf}, {"scaling": "other"},
    {"scaling": "parts"}, {"scaling": "parts", "original_length": 10, "low": 2.0, "high": 2.0},
    {"inv_freq": [1.0]}, {"inv_freq": [1.0] * 15 + [math.nan]},
    {"inv_freq": [1.0] * 16, "scaling": "linear"}, {"inv_freq": [1e300] * 16},
    {"base": 1e-300, "factor": 1e300, "scaling": "base"}])
def test_rotary_arguments(rbkv, args):
    with pytest.raises(ValueError):
        rbkv.Rotary(**{"rotary_dim": 32, "device": "cpu", **args})


def test_binding_checks(rbkv):
    cfg = rbkv.Config(8, 2, 64, 16, "f32", 33)
    t = rbkv.StepTables(cfg, 4, 8, 16, device="cpu")
    d = rbkv.StepDraft(t)
    assert d.place.shape == (16,) and d.ancestors.shape == (16, 4) and d.accepted.shape == (4,)
    with pytest.raises(AttributeError, match="cannot be replaced"):
        d.place = d.place.clone()
    with pytest.raises(AttributeError, match="cannot be deleted"):
        del d.path
    with pytest.raises(ValueError):                    # not on a GPU
        d.plan(torch.zeros(16, dtype=torch.int32))
    with pytest.raises(ValueError, match="is on meta"):
        d.accept(torch.zeros(16, dtype=torch.int32, device="meta"), None)
    other = rbkv.StepDraft(rbkv.StepTables(cfg, 4, 8, 16, device="cpu"))
    with pytest.raises(ValueError, match="other tables"):
        t._drafted(other)
    r = rbkv.Rotary(64, device="cpu")
    with pytest.raises(ValueError, match="rotary is on cpu"):
        r._on(torch.device("cuda", 0))


# ---- the oracle's pins ---------------------------------------------------------
def _built(seen, n_new, block, T, seed=0):
    rng = np.random.default_rng(seed)
    seen, n_new = np.asarray(seen), np.asarray(n_new)
    most = int((-(-(seen + n_new) // block)).max())
    blocks = int((-(-(seen + n_new) // block)).sum()) + 4
    table, free, _ = random_batch(rng, seen, block, most, blocks)
    st = oracle.step.build(seen, n_new, table, free, block, T)
    assert st.status == 0
    return st, blocks


def test_oracle_by_hand():
    """A tree of six tokens behind three cached ones (blocks of four), a chain
    of two, nothing."""
    st, _ = _built([3, 0, 5], [6, 2, 0], 4, 9)
    parent = [-1, 0, 0, 1, 2, 4, -1, 0, 7]
    p = D.plan(st, parent, 9)
    assert p.good and p.place.tolist() == [3, 4, 4, 5, 5, 6, 0, 1, -1]
    assert p.ancestors[:, 0].tolist() == [1, 3, 5, 11, 21, 53, 1, 3, 0]
    tokens = [10, 11, 12, 13, 14, 15, 20, 21, 0]
    chosen = [12, 13, 14, 0, 99, 0, 22, 7, 0]
    a = D.accept(st, parent, tokens, chosen, None, 4)
    assert a.path.tolist() == [0, 2, 4, -1, -1, -1, 6, -1, -1]
    assert a.accepted.tolist() == [3, 1, 0] and a.next_token.tolist() == [99, 22, -1]
    assert a.ctx.tolist() == [6, 1, 5]
    back = [i for i, (x, y) in enumerate(zip(st.free, a.free)) if x != y]
    assert back == [st.table[0, 2]]                  # tokens 8: the third block
    a = D.accept(st, parent, tokens, chosen, [4, 2, 1], 4)
    assert a.path.tolist() == [0, 1, 2, 3, -1, -1, 6, 7, -1] and a.accepted.tolist() == [4, 2, 0]
    cache = torch.arange(st.table.max() + 1.0)[:, None, None, None] * 4 + \
        torch.arange(4.0)[None, None, :, None]
    at = [cache[s // 4, 0, s % 4, 0].item() for s in st.slot[:6]]
    D.compact(st, D.accept(st, parent, tokens, chosen, None, 4), cache, 4)
    now = [cache[s // 4, 0, s % 4, 0].item() for s in st.slot[:6]]
    assert now == [at[0], at[2], at[4], *at[3:]]


def test_oracle_bad_trees_are_chains():
    st, _ = _built([0, 0, 0], [3, 2, 129], 16, 134)
    for parent in ([-1, 1, 0], [0, 0, 1], [-1, 0, -2], [-1, 0, 2]):
        p = D.plan(st, parent + [-1, -1] + D.chain(129), 134)
        assert not p.good and p.place[:5].tolist() == [0, 1, 2, 0, 0]
        assert p.ancestors[:5, 0].tolist() == [1, 3, 7, 1, 2]
    long = D.chain(129)
    long[100] = 3
    p = D.plan(st, [-1, 0, 0, -1, -1] + long, 134)
    assert not p.good and p.place[5:].tolist() == list(range(129)) and not p.ancestors[5:].any()


def test_reference_of_chains_is_the_causal_one():
    rng = np.random.default_rng(3)
    st, blocks = _built([5, 0, 20], [4, 1, 7], 8, 12)
    gen = torch.Generator().manual_seed(1)
    q = torch.randn(12, 4, 32, generator=gen)
    kc, vc = (torch.randn(blocks, 2, 8, 32, generator=gen) for _ in range(2))
    chains = np.array(D.chain(4) + D.chain(1) + D.chain(7))
    a = draft_reference(st, chains, q, kc, vc, [1, 2], 11)
    b = reference(st, q, kc, vc, [1, 2], 11)
    for x, y in zip(a, b):
        assert torch.allclose(x, y, rtol=1e-12, atol=1e-12)
    # a token sees what it would see if its path were all there is
    parent = random_trees(rng, [4, 1, 7], 12)
    full = draft_reference(st, parent, q, kc, vc, [], 0)[0]
    p, _ = D.parents_of(st, parent, 2)
    up = D.way_up(p, 6)
    slots = [st.table[2, x // 8] * 8 + x % 8 for x in list(range(20)) + [20 + j for j in up]]
    k, v = (torch.stack([c[s // 8, 1, s % 8] for s in slots]).double() for c in (kc, vc))
    w = torch.softmax(k @ q[11, 3].double() / math.sqrt(32), 0)
    assert torch.allclose(full[11, 3], w @ v, rtol=1e-12, atol=1e-12)


def test_oracle_rotation():
    rng = np.random.default_rng(4)
    x = rng.standard_normal((3, 2, 12))
    theta = np.array([1.0, 0.3, 0.01])
    for layout in ("half", "interleaved"):
        y = D.rotate(x, [0, 1, 1000], theta, layout, 2.0)
        assert np.allclose(y[0, :, :6], 2 * x[0, :, :6]) and np.array_equal(y[..., 6:], x[..., 6:])
        a, b = (0, 3) if layout == "half" else (0, 1)
        turned = (x[1, 0, a] + 1j * x[1, 0, b]) * np.exp(1j) * 2
        assert np.allclose([y[1, 0, a], y[1, 0, b]], [turned.real, turned.imag])
    # the angle between two rotated vectors goes by the distance of their positions
    u = D.rotate(x, [5, 5, 5], theta, "half")[..., :6]
    v = D.rotate(x, [9, 9, 9], theta, "half")[..., :6]
    u2 = D.rotate(x, [105, 105, 105], theta, "half")[..., :6]
    v2 = D.rotate(x, [109, 109, 109], theta, "half")[..., :6]
    assert np.allclose((u[0, 0] * v[1, 1]).sum(), (u2[0, 0] * v2[1, 1]).sum())
