"""Device-built steps without a GPU: argument checks of the C entries (refused
before anything is launched), the binding's checks, the oracle's own pins."""
import ctypes as C

import numpy as np
import pytest
import torch

import oracle
from step_harness import free_words, random_batch, reference

INVALID, UNSUPPORTED, WORKSPACE = -1, -5, -6
FAKE = 0x10000          # never dereferenced: every call below is refused


def _tables(rbkv, **change):
    t = rbkv._StepTables(4, 8, 16, *([FAKE] * 8))
    for k, v in change.items():
        setattr(t, k, v)
    return t


def _cfg(rbkv, hq=8, hkv=2, d=64, block=16, dtype="f32", blocks=32):
    return rbkv.Config(hq, hkv, d, block, dtype, blocks)._c()


def _build(rbkv, cfg=None, t=None, seen=FAKE, n_new=FAKE + 64, table=None, free=None):
    cfg, t = cfg or _cfg(rbkv), t or _tables(rbkv)
    return rbkv.lib().rbkv_step_build(C.byref(cfg), C.byref(t), seen, n_new, table, free, None)


@pytest.mark.parametrize("change", [
    {"num_seqs": 0}, {"num_seqs": -3}, {"max_blocks": 0}, {"max_tokens": 0},
    {"block_table": None}, {"free_words": None}, {"q_start": None}, {"ctx": None},
    {"position": None}, {"slot": None}, {"plan": None}, {"status": None},
    {"plan": FAKE + 2}, {"max_tokens": 2 ** 31 - 1}])
def test_bad_tables_are_refused(rbkv, change):
    t = _tables(rbkv, **change)
    L, cfg = rbkv.lib(), _cfg(rbkv)
    assert _build(rbkv, t=t) == INVALID
    assert L.rbkv_step_release(C.byref(cfg), C.byref(t), FAKE, None) == INVALID
    assert L.rbkv_step_append(C.byref(cfg), C.byref(t), FAKE, FAKE, FAKE, FAKE, None) == INVALID
    assert L.rbkv_step_attention(C.byref(cfg), C.byref(t), FAKE, FAKE, FAKE, None, 0, FAKE + 256,
                                 FAKE, 1 << 40, None) == INVALID
    assert b"" != L.rbkv_last_error()
    assert L.rbkv_step_workspace_bytes(C.byref(cfg), C.byref(t), 100) == 0


def test_bad_lengths_and_aliases_are_refused(rbkv):
    t = _tables(rbkv, ctx=FAKE + 512, q_start=FAKE + 1024)
    assert _build(rbkv, seen=None) == INVALID
    assert _build(rbkv, n_new=None) == INVALID
    assert _build(rbkv, seen=FAKE + 1) == INVALID
    assert _build(rbkv, t=t, n_new=FAKE + 512) == INVALID          # n_new = ctx
    assert _build(rbkv, t=t, seen=FAKE + 1024) == INVALID          # seen = q_start
    # seen = ctx with a table read from elsewhere: the copy would race with ctx
    assert _build(rbkv, t=t, seen=FAKE + 512, table=FAKE + 4096) == INVALID
    L, cfg = rbkv.lib(), _cfg(rbkv)
    assert L.rbkv_step_release(C.byref(cfg), C.byref(t), None, None) == INVALID
    assert L.rbkv_step_release(C.byref(cfg), C.byref(t), FAKE + 512, None) == INVALID
    assert L.rbkv_step_device_status(None, None) == INVALID
    assert L.rbkv_step_build(None, C.byref(t), FAKE, FAKE, None, None, None) == INVALID
    assert L.rbkv_step_build(C.byref(cfg), None, FAKE, FAKE, None, None, None) == INVALID


def test_bad_shapes_are_refused(rbkv):
    assert _build(rbkv, cfg=_cfg(rbkv, hq=8, hkv=3)) == INVALID
    assert _build(rbkv, cfg=_cfg(rbkv, d=48)) == UNSUPPORTED
    assert _build(rbkv, cfg=_cfg(rbkv, hq=65, hkv=1)) == UNSUPPORTED
    assert _build(rbkv, cfg=_cfg(rbkv, blocks=0)) == INVALID
    cfg, t = _cfg(rbkv, 64, 64, 256), _tables(rbkv, max_tokens=1 << 20)
    assert rbkv.lib().rbkv_step_append(C.byref(cfg), C.byref(t), FAKE, FAKE, FAKE, FAKE,
                                       None) == UNSUPPORTED


def test_attention_refusals(rbkv):
    L, cfg, t = rbkv.lib(), _cfg(rbkv), _tables(rbkv)

    def call(q=FAKE, k=FAKE, v=FAKE, ids=FAKE, n=5, o=FAKE + 4096, ws=FAKE, size=1 << 40):
        return L.rbkv_step_attention(C.byref(cfg), C.byref(t), q, k, v, ids, n, o, ws, size, None)

    for bad in ({"q": None}, {"k": None}, {"v": None}, {"o": None}, {"q": FAKE + 8},
                {"k": FAKE + 4}, {"v": FAKE + 2}, {"o": FAKE + 8}, {"n": -1},
                {"n": (1 << 30) + 1}, {"ids": None}, {"ids": FAKE + 2}, {"q": FAKE + 4096}, {"ws": FAKE + 16}):
        assert call(**bad) == INVALID, bad


def test_workspace_is_checked_where_one_is_needed(rbkv):
    L, t = rbkv.lib(), _tables(rbkv, max_tokens=64)
    cfg = _cfg(rbkv, 8, 2, 128, 64, "bf16")
    need = L.rbkv_step_workspace_bytes(C.byref(cfg), C.byref(t), 1000)
    if need:
        for ws, size in ((None, 0), (FAKE, need - 1)):
            assert L.rbkv_step_attention(C.byref(cfg), C.byref(t), FAKE, FAKE, FAKE, FAKE, 1000,
                                         FAKE + 4096, ws, size, None) == WORKSPACE


def test_plan_size(rbkv):
    L = rbkv.lib()
    assert L.rbkv_step_plan_ints(0, 5) == 0 and L.rbkv_step_plan_ints(5, 0) == 0
    assert L.rbkv_step_plan_ints(1, 1) > 0
    assert L.rbkv_step_plan_ints(70000, 70000) > 4 * 70000


def test_binding_checks(rbkv):
    cfg = rbkv.Config(8, 2, 64, 16, "f32", 33)
    with pytest.raises(ValueError):
        rbkv.StepTables(cfg, 0, 8, 16, device="cpu")
    with pytest.raises(ValueError):
        rbkv.StepTables(cfg, 4, 8, 0, device="cpu")
    with pytest.raises(ValueError):
        rbkv.StepTables(rbkv.Config(8, 2, 64, 16, "f32", 0), 4, 8, 16, device="cpu")
    t = rbkv.StepTables(cfg, 4, 8, 16, device="cpu")
    assert t.free.tolist() == [-1, 1]            # 33 blocks: the second word holds one
    with pytest.raises(ValueError):              # not on a GPU
        t._ptr(torch.zeros(4, dtype=torch.int32), "seen", torch.int32, (4,))
    other = torch.zeros(4, dtype=torch.int32, device="meta")
    with pytest.raises(ValueError, match="is on meta"):
        t._ptr(other, "seen", torch.int32, (4,))
    with pytest.raises(ValueError, match="prefix_table"):
        t.attention(None, None, None, prefix_table=torch.zeros(2, dtype=torch.int32),
                    prefix_len=33)


def test_free_words_match_the_binding(rbkv):
    for n in (1, 31, 32, 33, 64, 100):
        t = rbkv.StepTables(rbkv.Config(8, 2, 64, 16, "f32", n), 1, 1, 1, device="cpu")
        assert t.free.tolist() == free_words(np.ones(n, bool)).tolist()


# ---- the oracle's pins ---------------------------------------------------------
def test_oracle_step_by_hand():
    table = np.full((3, 3), -1)
    table[0, 0], table[2, :2] = 5, [1, 7]
    free = [True, False, True, True, True, False, True, False]
    st = oracle.step.build([3, 0, 8], [2, 0, 1], table, free, 4, 4)
    assert st.status == 0 and st.q_start.tolist() == [0, 2, 2, 3] and st.ctx.tolist() == [5, 0, 9]
    assert st.table.tolist() == [[5, 0, -1], [-1, -1, -1], [1, 7, 2]]
    assert st.position.tolist() == [3, 4, 8, -1] and st.slot.tolist() == [23, 0, 8, -1]
    assert st.free == [False, False, False, True, True, False, True, False]


@pytest.mark.parametrize("seen,n_new,status", [
    ([3, -1], [1, 1], -1), ([3, 1], [1, -2], -1), ([0, 0], [5, 4], -6), ([12, 0], [1, 0], -6),
    ([0, 0], [5, 1], -2)])
def test_oracle_step_that_does_not_fit(seen, n_new, status):
    table, free = np.full((2, 3), -1), [True, False, True]
    st = oracle.step.build(seen, n_new, table, free, 4, 8)
    assert st.status == status and st.q_start.tolist() == [0, 0, 0]
    assert st.ctx.tolist() == seen and st.free == free and (st.slot == -1).all()


def test_oracle_agrees_with_the_composer():
    """The same lengths, composed on the host: the same ids and slots."""
    lens = [5, 40, 17, 1]
    comp = oracle.Composer(16, 64)
    m0 = comp.compose(10 ** 6, 0, [(i, n, 0) for i, n in enumerate(lens)])
    st = oracle.step.build([0] * 4, lens, np.full((4, 8), -1), [True] * 64, 16, sum(lens))
    assert st.slot.tolist() == list(m0.slot) and st.q_start.tolist() == list(m0.q_start)
    m1 = comp.compose(10 ** 6, 0, [(i, n, n) for i, n in enumerate(lens)])
    st = oracle.step.build(lens, [1] * 4, st.table, st.free, 16, 4)
    assert st.slot.tolist() == list(m1.slot) and st.ctx.tolist() == list(m1.ctx)


@pytest.mark.parametrize("prefix", [0, 1, 16, 37])
def test_reference_and_oracle_attention(prefix):
    """The vectorised reference equals the loops; a prefix equals the same
    tokens at the head of every sequence; one key gives its value."""
    rng = np.random.default_rng(prefix)
    B, H_q, H_kv, D = 8, 4, 2, 32
    seen, n_new = [0, 9, 3, 0], [1, 2, 0, 13]
    pre_blocks = -(-prefix // B)
    table, free, ids = random_batch(rng, seen, B, 4, 40, pre_blocks)
    st = oracle.step.build(seen, n_new, table, free, B, 20)
    kc, vc = (torch.randn(40, H_kv, B, D, dtype=torch.float64) for _ in range(2))
    q = torch.randn(20, H_q, D, dtype=torch.float64)
    ref = reference(st, q, kc, vc, ids, prefix)[0]
    loops = oracle.step.attention(st, q.numpy(), kc.numpy(), vc.numpy(), ids, prefix)
    assert np.abs(ref.numpy() - loops).max() < 1e-12
    if prefix == 0:
        assert torch.allclose(ref[0], vc[st.table[0, 0], :, 0].repeat_interleave(2, 0))
    if prefix % B == 0 and prefix:
        # the prefix's blocks as the head of a longer table
        whole = np.concatenate([np.tile(ids, (4, 1)), st.table], 1)
        moved = oracle.step.Step(0, st.q_start, st.ctx + prefix, whole, [], st.position + prefix,
                                 st.slot)
        assert torch.allclose(reference(moved, q, kc, vc, [], 0)[0], ref, atol=1e-12)


def test_a_strided_workspace_is_refused(rbkv):
    """Its bytes are not the ones behind its address (an expanded one has one)."""
    cfg = rbkv.Config(8, 2, 64, 16, "f32", 33)
    t = rbkv.StepTables(cfg, 4, 8, 16, device="cpu")
    t._index = -1                                # (a CPU tensor's: past the device check)
    for ws in (torch.empty(1, dtype=torch.uint8).expand(1 << 20),
               torch.empty(1 << 10, 2, dtype=torch.uint8)[:, 0]):
        with pytest.raises(ValueError, match="contiguous"):
            t.attention(None, None, None, o=torch.empty(0), workspace=ws)


@pytest.mark.parametrize("sizes", [(2 ** 32 + 4, 8, 16), (4, 2 ** 32 + 8, 16), (4, 8, 2 ** 32 + 16),
                                   (2 ** 31, 8, 16), (4, 8, 2 ** 31)])
def test_sizes_past_32_bits_are_refused(rbkv, sizes):
    """(meta: nothing is allocated where they were taken for small ones)"""
    cfg = rbkv.Config(8, 2, 64, 16, "f32", 33)
    with pytest.raises(ValueError, match="32 bits"):
        rbkv.StepTables(cfg, *sizes, device="meta")


@pytest.mark.parametrize("prefix_len", [2 ** 32, 2 ** 31, -2 ** 32 + 5])
def test_prefix_lengths_past_32_bits_are_refused(rbkv, prefix_len):
    t = rbkv.StepTables(rbkv.Config(8, 2, 64, 16, "f32", 33), 4, 8, 16, device="cpu")
    with pytest.raises(ValueError, match="32 bits"):
        t.workspace_bytes(prefix_len)
    with pytest.raises(ValueError, match="32 bits"):
        t.attention(None, None, None, prefix_len=prefix_len, o=torch.empty(0),
                    workspace=torch.empty(0))


def test_the_arrays_cannot_be_replaced(rbkv):
    """The library holds their addresses: another tensor under the name would
    not be used, and would free the memory that is."""
    t = rbkv.StepTables(rbkv.Config(8, 2, 64, 16, "f32", 33), 4, 8, 16, device="cpu")
    for name in ("block_table", "free", "q_start", "ctx", "position", "slot", "plan", "status"):
        held = getattr(t, name)
        with pytest.raises(AttributeError):
            setattr(t, name, held.clone())
        assert getattr(t, name) is held
    t.free &= 1                                  # in place: the same tensor
    assert t.free.tolist() == [1, 1]
    before = t.ctx
    t.ctx += 3
    assert t.ctx is before and t.ctx.tolist() == [3, 3, 3, 3]
    for name in ("free", "ctx"):
        with pytest.raises(AttributeError):
            delattr(t, name)


def _apart(rbkv, S=4, max_blocks=8, T=16):
    """Tables whose arrays lie a megabyte apart, and addresses that are free."""
    at = [FAKE + (i << 20) for i in range(12)]
    return rbkv._StepTables(S, max_blocks, T, *at[:8]), at[8:]


# (a table array, bytes into it): where an input would be overwritten by the step
OVERLAPS = [("q_start", 4), ("q_start", 16), ("ctx", 4), ("ctx", -12), ("position", 0),
            ("position", 60), ("slot", 8), ("plan", 16), ("status", 12), ("free_words", 0),
            ("block_table", 124)]


@pytest.mark.parametrize("name,at", OVERLAPS)
def test_inputs_that_a_step_would_overwrite_are_refused(rbkv, name, at):
    t, (a, b, c, d) = _apart(rbkv)
    where = getattr(t, name) + at
    for args in ((where, a), (a, where)):
        assert _build(rbkv, t=t, seen=args[0], n_new=args[1]) == INVALID
        assert b"overlap" in rbkv.lib().rbkv_last_error()
    if name != "free_words" and at >= 0:                     # (one word of free bits)
        assert _build(rbkv, t=t, seen=a, n_new=b, free=where) == INVALID
        assert b"overlap" in rbkv.lib().rbkv_last_error()
    assert _build(rbkv, t=t, seen=a, n_new=b, table=where) == INVALID
    assert b"overlap" in rbkv.lib().rbkv_last_error()
    cfg = _cfg(rbkv)
    if name in ("ctx", "free_words", "status"):
        assert rbkv.lib().rbkv_step_release(C.byref(cfg), C.byref(t), where, None) == INVALID
        assert b"overlap" in rbkv.lib().rbkv_last_error()


def test_arrays_in_place_are_not_overlaps(rbkv):
    """(without a GPU the launch fails: any other status than INVALID will do)"""
    t, (a, b, c, d) = _apart(rbkv)
    if torch.cuda.is_available():
        pytest.skip("would launch with made-up addresses")
    for kw in ({"seen": t.ctx, "n_new": a}, {"seen": a, "n_new": a},
               {"seen": t.ctx, "n_new": b, "table": t.block_table, "free": t.free_words},
               {"seen": t.ctx + 16, "n_new": t.ctx - 16},              # next to it
               {"seen": a, "n_new": b, "table": c, "free": d}):
        assert _build(rbkv, t=t, **kw) != INVALID, kw
