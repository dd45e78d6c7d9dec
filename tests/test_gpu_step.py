"""Steps built on the GPU from device-side lengths: tables, slots, append and
shared-prefix attention against the oracle, refusals, captured graphs."""
import numpy as np
import pytest
import torch

import oracle
from step_harness import error_bound, free_words, i32, random_batch, reference

pytestmark = pytest.mark.gpu

NO_BLOCKS, INVALID, WORKSPACE, BOUNDS = -2, -1, -6, -4


def _cfg(rbkv, hq=8, hkv=2, d=64, block=16, dtype="f32", blocks=64):
    return rbkv.Config(hq, hkv, d, block, dtype, blocks)


def _equal(t, want: oracle.step.Step):
    assert t.q_start.tolist() == want.q_start.tolist()
    assert t.ctx.tolist() == want.ctx.tolist()
    assert np.array_equal(t.block_table.cpu().numpy(), want.table)
    assert np.array_equal(t.free.cpu().numpy(), free_words(want.free))
    assert np.array_equal(t.position.cpu().numpy(), want.position)
    assert np.array_equal(t.slot.cpu().numpy(), want.slot)


# ---- tables --------------------------------------------------------------------
TABLES = [
    # seqs, longest, most new tokens, block, spare blocks, spare rows
    (1, 0, 1, 16, 1, 0), (1, 5, 1, 1, 3, 2), (3, 40, 0, 8, 0, 5), (17, 300, 1, 64, 9, 0),
    (33, 90, 7, 16, 100, 12), (100, 1000, 3, 128, 31, 1), (513, 700, 1, 16, 1000, 0),
    (7, 50, 900, 16, 5, 3), (400, 9000, 2, 16, 200000, 3), (1500, 30, 3, 16, 70, 4),
    (4100, 60, 2, 16, 40000, 77), (9000, 3, 1, 5, 20, 1)]


@pytest.mark.parametrize("S,longest,most,block,spare,rows", TABLES)
@pytest.mark.parametrize("in_place", [True, False])
def test_tables_against_oracle(rbkv, S, longest, most, block, spare, rows, in_place):
    rng = np.random.default_rng(S * 31 + longest)
    seen = rng.integers(0, longest + 1, S)
    n_new = rng.integers(0, most + 1, S)
    if S > 2:
        n_new[rng.integers(0, S, S // 3)] = 0
    max_blocks = -(-(longest + most) // block) + 1
    grow = (-(-(seen + n_new) // block) - -(-seen // block)).sum()
    blocks = int((-(-seen // block)).sum() + grow + spare) or 1
    table, free, _ = random_batch(rng, seen, block, max_blocks, blocks)
    T = max(1, int(n_new.sum()) + rows)
    want = oracle.step.build(seen, n_new, table, free, block, T)
    assert want.status == 0
    t = rbkv.StepTables(_cfg(rbkv, block=block, blocks=blocks), S, max_blocks, T)
    src, bits = i32(table), i32(free_words(free))
    if in_place:
        t.block_table.copy_(src)
        t.free.copy_(bits)
        t.ctx.copy_(i32(seen))
        t.build(t.ctx, i32(n_new))
    else:
        t.build(i32(seen), i32(n_new), block_table=src, free=bits)
        assert np.array_equal(src.cpu().numpy(), table)      # the inputs stay
        assert np.array_equal(bits.cpu().numpy(), free_words(free))
    _equal(t, want)
    t.device_status()


@pytest.mark.parametrize("S", [40, 1500])
@pytest.mark.parametrize("in_place", [True, False])
def test_captured_tables(rbkv, S, in_place):
    """A captured build and release, replayed over other lengths (one CTA, and
    a cluster)."""
    rng = np.random.default_rng(S)
    B, max_blocks, T, blocks = 8, 12, 3 * S, 9 * S
    t = rbkv.StepTables(_cfg(rbkv, block=B, blocks=blocks), S, max_blocks, T)
    seen, n_new, done = (torch.zeros(S, dtype=torch.int32, device="cuda") for _ in range(3))
    src, bits = torch.empty_like(t.block_table), torch.empty_like(t.free)

    def step():
        t.build(seen, n_new, **({} if in_place else {"block_table": src, "free": bits}))
        t.release(done)

    step()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(4):
        lengths, new = rng.integers(0, 60, S), rng.integers(0, 4, S)
        table, free, _ = random_batch(rng, lengths, B, max_blocks, blocks)
        seen.copy_(i32(lengths))
        n_new.copy_(i32(new))
        for mine, given, value in ((t.block_table, src, table), (t.free, bits, free_words(free))):
            (mine if in_place else given).copy_(i32(value))
        gone = rng.random(S) < 0.3
        done.copy_(i32(gone))
        graph.replay()
        want = oracle.step.build(lengths, new, table, free, B, T)
        assert want.status == 0
        for s in np.flatnonzero(gone):
            for c in range(-(-int(want.ctx[s]) // B)):
                want.free[want.table[s, c]] = True
        want.ctx[gone] = 0
        _equal(t, want)
    t.device_status()


@pytest.mark.parametrize("seen,n_new,T,status", [
    ([3, -1, 5], [1, 1, 1], 8, INVALID), ([3, 1, 0], [1, -2, 1], 8, INVALID),
    ([0, 0, 0], [5, 4, 0], 8, WORKSPACE), ([12, 0, 0], [1, 0, 0], 8, WORKSPACE),
    ([0, 0, 0], [2 ** 31 - 1, 2 ** 31 - 1, 3], 8, WORKSPACE),
    ([2 ** 31 - 1, 0, 0], [2 ** 31 - 1, 0, 0], 8, WORKSPACE), ([4, 0, 4], [1, 1, 1], 8, NO_BLOCKS)])
@pytest.mark.parametrize("in_place", [True, False])
def test_a_step_that_does_not_fit_is_empty(rbkv, seen, n_new, T, status, in_place):
    table = np.array([[7, 3, -1], [-1, -1, -1], [2, -1, -1]])
    free = [False, True, False, False, True, False, False, False]
    t = rbkv.StepTables(_cfg(rbkv, block=4, blocks=8), 3, 3, T)
    q = torch.randn(T, 8, 64, device="cuda")
    kc, vc = torch.randn(8, 2, 4, 64, device="cuda"), torch.randn(8, 2, 4, 64, device="cuda")
    before = kc.clone()
    if in_place:
        t.block_table.copy_(i32(table))
        t.free.copy_(i32(free_words(free)))
        t.build(i32(seen), i32(n_new))
    else:
        t.build(i32(seen), i32(n_new), block_table=i32(table), free=i32(free_words(free)))
    assert t.q_start.tolist() == [0, 0, 0, 0] and t.ctx.tolist() == seen
    assert np.array_equal(t.block_table.cpu().numpy(), table)
    assert np.array_equal(t.free.cpu().numpy(), free_words(free))
    assert (t.position == -1).all() and (t.slot == -1).all()
    o = torch.full_like(q, 3.0)
    t.append(torch.randn(T, 2, 64, device="cuda"), torch.randn(T, 2, 64, device="cuda"), kc, vc)
    t.attention(q, kc, vc, prefix_table=i32([0]), prefix_len=4, o=o)
    assert torch.equal(kc, before) and (o == 3.0).all()
    with pytest.raises(rbkv.RbkvError) as e:
        t.device_status()
    assert e.value.status == status
    t.device_status()                                    # reading cleared it
    t.build(i32([0, 0, 0]), i32([1, 0, 1]))              # the tables still work
    assert t.q_start.tolist() == [0, 1, 1, 2]
    t.device_status()


def test_bad_block_ids_in_a_table_are_reported(rbkv):
    t = rbkv.StepTables(_cfg(rbkv, block=4, blocks=8), 2, 3, 4)
    t.build(i32([2, 5]), i32([1, 1]), block_table=i32([[99, -1, -1], [1, -7, -1]]))
    assert t.slot.tolist() == [-1, -1, -1, -1] and t.position.tolist() == [2, 5, -1, -1]
    with pytest.raises(rbkv.RbkvError) as e:
        t.device_status()
    assert e.value.status == BOUNDS
    t.ctx.copy_(i32([3, 6]))
    t.free.zero_()
    t.release(i32([1, 1]))
    assert t.free.tolist() == [1 << 1] and t.ctx.tolist() == [0, 0]
    with pytest.raises(rbkv.RbkvError):
        t.device_status()


def test_a_serving_loop_of_steps(rbkv):
    """Sixty steps in place: requests come, grow by ragged amounts, finish and
    give their blocks back; every step against the oracle."""
    rng = np.random.default_rng(5)
    S, B, blocks, max_blocks, T = 13, 8, 150, 12, 64
    t = rbkv.StepTables(_cfg(rbkv, block=B, blocks=blocks), S, max_blocks, T)
    ctx, table, free = np.zeros(S, np.int64), np.full((S, max_blocks), -1), [True] * blocks
    for _ in range(60):
        n_new = rng.choice([0, 1, 1, 1, 2, 17], S)
        n_new = np.minimum(n_new, max_blocks * B - ctx)
        while n_new.sum() > T:
            n_new[np.argmax(n_new)] = 1
        want = oracle.step.build(ctx, n_new, table, free, B, T)
        assert want.status == 0
        t.build(t.ctx, i32(n_new))
        _equal(t, want)
        ctx, table, free = want.ctx, want.table, want.free
        done = (rng.random(S) < 0.1) | (ctx > 80)
        for s in np.flatnonzero(done):
            for c in range(-(-ctx[s] // B)):
                free[table[s, c]] = True
            ctx[s] = 0
        t.release(i32(done))
        assert np.array_equal(t.free.cpu().numpy(), free_words(free))
        assert t.ctx.tolist() == ctx.tolist()
    t.device_status()


# ---- append and attention --------------------------------------------------------
def _case(rbkv, hq, hkv, D, block, dtype, prefix, seen, n_new, pad=0, seed=0, fill=None,
          scale=1.0, change=None):
    """A built and appended step with its caches; `fill` in every slot that no
    token has written (the step's own rows are written by the append);
    `change(q, k_new, v_new)` may alter the step's rows first."""
    rng = np.random.default_rng(seed)
    seen, n_new = np.asarray(seen), np.asarray(n_new)
    S = len(seen)
    max_blocks = int((-(-(seen + n_new) // block)).max()) + 1
    pre_blocks = -(-prefix // block)
    blocks = int((-(-(seen + n_new) // block)).sum()) + pre_blocks + 3
    table, free, ids = random_batch(rng, seen, block, max_blocks, blocks, pre_blocks)
    T = max(1, int(n_new.sum()) + pad)
    want = oracle.step.build(seen, n_new, table, free, block, T)
    assert want.status == 0
    cfg = _cfg(rbkv, hq, hkv, D, block, dtype, blocks)
    dt = cfg.torch_dtype
    gen = torch.Generator().manual_seed(seed)

    def normal(*shape):
        return (torch.randn(*shape, generator=gen) * scale).to(dt)

    kc, vc = normal(*cfg.cache_shape()), normal(*cfg.cache_shape())
    if fill is not None:
        live = torch.zeros(blocks, block, dtype=torch.bool)
        for s in range(S):
            for p in range(int(seen[s])):
                live[table[s, p // block], p % block] = True
        for p in range(prefix):
            live[ids[p // block], p % block] = True
        kc[~live[:, None].expand(-1, hkv, -1)] = fill
        vc[~live[:, None].expand(-1, hkv, -1)] = fill
    q, kn, vn = normal(T, hq, D), normal(T, hkv, D), normal(T, hkv, D)
    if change is not None:
        change(q, kn, vn)
    t = rbkv.StepTables(cfg, S, max_blocks, T)
    t.build(i32(seen), i32(n_new), block_table=i32(table), free=i32(free_words(free)))
    kd, vd = kc.cuda(), vc.cuda()
    t.append(kn.cuda(), vn.cuda(), kd, vd)
    rows = int(want.q_start[-1])
    for r in range(rows):
        b, off = divmod(int(want.slot[r]), block)
        kc[b, :, off], vc[b, :, off] = kn[r], vn[r]
    return t, want, q, kd, vd, kc, vc, ids, rows


def _check(rbkv, hq, hkv, D, block, dtype, prefix, seen, n_new, pad=0, seed=0, fill=None,
           scale=1.0):
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, hq, hkv, D, block, dtype, prefix, seen,
                                                  n_new, pad, seed, fill, scale)
    nan = torch.equal(kd.cpu().view(torch.uint8), kc.view(torch.uint8))
    assert nan and torch.equal(vd.cpu().view(torch.uint8), vc.view(torch.uint8))
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    t.attention(q.cuda(), kd, vd, prefix_table=i32(ids) if prefix else None, prefix_len=prefix,
                o=o)
    t.device_status()
    o = o.cpu()
    assert (o[rows:] == 7.0).all()                     # rows past the step's are left alone
    if fill is not None:
        kc, vc = (torch.nan_to_num(x.float(), 0, 0, 0) for x in (kc, vc))
    ref = reference(want, q, kc, vc, ids, prefix)
    err = (o[:rows].double() - ref[0]).abs()
    bound = error_bound(ref, D, dtype)
    assert torch.isfinite(o).all()
    assert (err <= bound).all(), float((err / bound).max())
    return t, o


MIXED = ([0, 0, 5, 63, 64, 200, 17, 0, 31, 130], [1, 40, 1, 1, 1, 1, 0, 3, 33, 7])

SHAPES = [(8, 2, 64, 16, "f32"), (4, 4, 32, 5, "f32"), (3, 1, 256, 16, "f32"),
          (8, 2, 64, 16, "bf16"), (6, 2, 96, 24, "bf16"), (32, 32, 128, 64, "bf16"),
          (32, 8, 128, 64, "bf16"), (16, 2, 128, 16, "bf16"), (10, 2, 128, 32, "bf16"),
          (16, 1, 128, 128, "bf16"), (40, 2, 128, 64, "bf16"), (64, 1, 128, 8, "bf16"),
          (8, 8, 128, 192, "bf16"), (7, 1, 128, 256, "bf16"), (12, 1, 128, 40, "bf16")]


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("prefix", [0, 1, 100, 333])
def test_attention_mixed_steps(rbkv, shape, prefix):
    _check(rbkv, *shape, prefix, *MIXED, pad=9, seed=prefix + shape[0])


@pytest.mark.parametrize("shape", [(8, 2, 64, 16, "f32"), (32, 8, 128, 64, "bf16"),
                                   (8, 8, 128, 16, "bf16")], ids=str)
@pytest.mark.parametrize("prefix", [0, 63, 64, 65, 127, 128, 129, 1000])
@pytest.mark.parametrize("own", [1, 2, 16, 63, 64, 65, 128, 129])
def test_attention_borders_of_tiles(rbkv, shape, prefix, own):
    """Lengths at the borders of blocks and key tiles, every unwritten slot NaN."""
    _check(rbkv, *shape, prefix, [own - 1, 0, max(0, own - 3)], [1, own, min(own, 3)], seed=own,
           fill=float("nan"))


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (8, 2, 64, 16, "f32")], ids=str)
@pytest.mark.parametrize("fill", [float("inf"), -3.0e38, float("nan")])
def test_unwritten_slots_do_not_matter(rbkv, shape, fill):
    _check(rbkv, *shape, 77, *MIXED, pad=3, fill=fill)


# (sequence, token, value) of the step below: non-finite values of new tokens
POKES = [(0, 0, float("inf")), (0, 150, float("nan")), (0, 299, float("-inf")),
         (1, 1, float("nan")), (1, 2, float("inf")), (2, 0, float("inf")),
         (3, 20, float("inf")), (3, 21, float("-inf")), (4, 7, float("inf")),
         (4, 15, float("nan"))]
POKED = ([70, 0, 5, 130, 1000, 9], [300, 3, 1, 40, 16, 1])


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (8, 8, 128, 16, "bf16"),
                                   (8, 4, 128, 8, "bf16"), (16, 1, 128, 128, "bf16"),
                                   (8, 2, 64, 16, "bf16"), (8, 2, 32, 5, "f32")], ids=str)
@pytest.mark.parametrize("prefix", [0, 200])
def test_later_values_do_not_reach_earlier_rows(rbkv, shape, prefix):
    """Infinities and NaN in V of new tokens: the rows that see them have them
    at that head dim, every other element is what it is without them."""
    hq, hkv, D, block, dtype = shape
    starts = np.concatenate([[0], np.cumsum(POKED[1])])

    def change(q, kn, vn):
        for i, (s, tok, value) in enumerate(POKES):
            vn[starts[s] + tok, i % hkv, 3 * i:3 * i + 2] = value
        vn[starts[4] + 9, 0] = float("nan")              # a whole row

    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, prefix, *POKED, pad=5, seed=3,
                                                  change=change)
    o = t.attention(q.cuda(), kd, vd, prefix_table=i32(ids) if prefix else None,
                    prefix_len=prefix).cpu()[:rows].double()
    t.device_status()
    g = hq // hkv
    added = torch.zeros(rows, hq, D, dtype=torch.float64)
    for s in range(len(POKED[0])):
        a, b = int(starts[s]), int(starts[s + 1])
        for r in range(a, b):
            block_of, off = divmod(int(want.slot[r]), block)
            v = vc[block_of, :, off].double()
            v = torch.where(torch.isfinite(v), 0.0, v).repeat_interleave(g, 0)
            added[r:b] += v
    finite_v = torch.where(torch.isfinite(vc), vc, torch.zeros((), dtype=vc.dtype))
    ref = reference(want, q, kc, finite_v, ids, prefix)
    finite = added == 0
    err = (o - ref[0]).abs()
    assert (err[finite] <= error_bound(ref, D, dtype)[finite]).all()
    assert torch.equal(torch.isnan(o), torch.isnan(added))
    infinite = torch.isinf(added)
    assert torch.equal(o[infinite], added[infinite]) and 0 < int(infinite.sum())


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (8, 8, 128, 16, "bf16"),
                                   (8, 2, 32, 5, "f32")], ids=str)
@pytest.mark.parametrize("prefix", [0, 200])
def test_a_nan_key_or_query_reaches_its_rows_only(rbkv, shape, prefix):
    hq, hkv, D, block, dtype = shape
    starts = np.concatenate([[0], np.cumsum(POKED[1])])
    g = hq // hkv
    bad = torch.zeros(int(starts[-1]), hq, dtype=torch.bool)
    for s, tok in [(0, 130), (1, 1), (3, 39), (4, 8)]:
        bad[starts[s] + tok:starts[s + 1], g:2 * g] = True      # those who see key head 1
    bad[starts[5], 0] = bad[starts[0] + 17, 1] = True           # queries

    def change(q, kn, vn):
        for s, tok in [(0, 130), (1, 1), (3, 39), (4, 8)]:
            kn[starts[s] + tok, 1, 5] = float("nan")
        q[starts[5], 0, 2] = q[starts[0] + 17, 1, D - 1] = float("nan")

    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, prefix, *POKED, pad=5, seed=4,
                                                  change=change)
    o = t.attention(q.cuda(), kd, vd, prefix_table=i32(ids) if prefix else None,
                    prefix_len=prefix).cpu()[:rows].double()
    t.device_status()
    assert torch.isnan(o[bad]).all()
    clean = [torch.nan_to_num(x.float()).to(x.dtype) for x in (q, kc)]
    ref = reference(want, clean[0], clean[1], vc, ids, prefix)
    err = (o - ref[0]).abs()
    assert (err[~bad] <= error_bound(ref, D, dtype)[~bad]).all()


@pytest.mark.parametrize("hq,hkv,decodes,prefix,own", [
    (32, 8, 300, 700, 90), (32, 32, 40, 500, 30), (64, 8, 64, 2000, 300), (32, 8, 1, 5000, 400),
    (8, 1, 3, 4000, 1), (32, 8, 1, 1, 1), (64, 4, 130, 260, 40)])
def test_attention_decoding_batches(rbkv, hq, hkv, decodes, prefix, own):
    rng = np.random.default_rng(decodes)
    _check(rbkv, hq, hkv, 128, 64, "bf16", prefix, rng.integers(0, own, decodes),
           np.ones(decodes, int), seed=decodes)


@pytest.mark.parametrize("prefix", [0, 450])
def test_attention_prompt_chunks(rbkv, prefix):
    """Chunks of several hundred rows behind their own cached tokens."""
    _check(rbkv, 32, 8, 128, 64, "bf16", prefix, [0, 300, 64, 900], [700, 129, 257, 1], pad=40)
    _check(rbkv, 8, 8, 128, 16, "bf16", prefix, [500, 0], [300, 500])


@pytest.mark.parametrize("scale", [3.0, 30.0])
def test_attention_sharp_scores(rbkv, scale):
    """Scores far apart: the running maximum rises many times."""
    _check(rbkv, 32, 8, 128, 64, "bf16", 200, *MIXED, scale=scale)
    _check(rbkv, 8, 2, 64, 16, "f32", 200, *MIXED, scale=scale)


def test_rising_scores_in_both_parts(rbkv):
    """Every key scores higher than the one before, in the prefix and behind it."""
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, 8, 2, 128, 64, "bf16", 300,
                                                  [200, 0], [1, 60])
    q[:] = 1.0
    for i, (table, n) in enumerate(((ids, 300), (want.table[0], 201), (want.table[1], 60))):
        for p in range(n):
            kc[table[p // 64], :, p % 64] = 0.01 * (p + 300 * (i > 0))
    o = t.attention(q.cuda(), kc.cuda(), vd, prefix_table=i32(ids), prefix_len=300)
    ref = reference(want, q, kc, vc, ids, 300)
    err = (o.cpu().double() - ref[0]).abs()
    assert (err <= error_bound(ref, 128, "bf16")).all()


def test_repeats_are_bit_identical(rbkv):
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, 32, 8, 128, 64, "bf16", 900, *MIXED)
    ws = torch.empty(max(256, t.workspace_bytes(900)), dtype=torch.uint8, device="cuda")
    first = t.attention(q.cuda(), kd, vd, prefix_table=i32(ids), prefix_len=900, workspace=ws)
    for fill in (0, 255):                    # whatever the workspace held
        ws.fill_(fill)
        again = t.attention(q.cuda(), kd, vd, prefix_table=i32(ids), prefix_len=900, workspace=ws)
        assert torch.equal(first, again)


@pytest.mark.parametrize("hq,hkv,T", [(16, 1, 1), (17, 1, 1), (8, 1, 2), (9, 1, 2), (64, 1, 1),
                                      (4, 4, 16), (4, 4, 17), (64, 1, 3)])
@pytest.mark.parametrize("prefix", [0, 400])
def test_steps_around_sixteen_packed_rows(rbkv, hq, hkv, T, prefix):
    """Where the prefix goes from the streaming kernel to the tile kernel; the
    rows as single tokens and as one sequence's."""
    _check(rbkv, hq, hkv, 128, 32, "bf16", prefix, [40 + 3 * i for i in range(T)], [1] * T)
    _check(rbkv, hq, hkv, 128, 32, "bf16", prefix, [40, 0], [T, 0], seed=1)


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (4, 4, 128, 16, "bf16"),
                                   (8, 2, 64, 16, "f32")], ids=str)
def test_a_step_of_idle_slots_writes_nothing(rbkv, shape):
    for pad in (3, 40):                          # few rows and many
        t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 70, [5, 0, 300], [0, 0, 0],
                                                      pad=pad)
        assert rows == 0
        o = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
        t.attention(q.cuda(), kd, vd, prefix_table=i32(ids), prefix_len=70, o=o)
        t.device_status()
        assert (o == 7.0).all()


def test_attention_of_many_sequences(rbkv):
    """Tables of thousands of sequences (several CTAs build them), with prompts
    among the single tokens and idle slots."""
    rng = np.random.default_rng(9)
    n_new = rng.choice([0, 1, 1, 1, 3], 2100)
    n_new[[5, 700, 2099]] = [180, 65, 33]
    _check(rbkv, 4, 1, 128, 16, "bf16", 130, rng.integers(0, 40, 2100), n_new, pad=5)
    _check(rbkv, 2, 1, 32, 16, "f32", 30, rng.integers(0, 20, 2100), np.minimum(n_new, 3), pad=5)


@pytest.mark.parametrize("dtype,D", [("bf16", 128), ("f32", 64)])
def test_blocks_far_into_a_large_cache(rbkv, dtype, D):
    """Offsets past 2^31 elements: a step whose blocks lie at the end of the
    cache against the same step at the start of a small one."""
    hq, hkv, B, P, S = 16, 8, 64, 150, 4
    seen, n_new = np.array([70, 0, 200, 5]), np.array([1, 90, 1, 3])
    T, held, max_blocks = int(n_new.sum()), -(-(seen + n_new) // B), 5
    gen = torch.Generator().manual_seed(1)
    outs, far = [], (1 << 31) // (hkv * B * D) + 100
    for first in (0, far):
        cfg = _cfg(rbkv, hq, hkv, D, B, dtype, first + 20)
        dt = cfg.torch_dtype
        kc, vc = (torch.empty(cfg.cache_shape(), dtype=dt, device="cuda") for _ in range(2))
        assert first == 0 or kc.numel() > 1 << 31
        gen.manual_seed(1)
        for c in (kc, vc):
            c[first:] = torch.randn(20, hkv, B, D, generator=gen).to(dt).cuda()
        q, kn, vn = (torch.randn(T, h, D, generator=gen).to(dt).cuda() for h in (hq, hkv, hkv))
        table = np.full((S, max_blocks), -1)
        free = np.zeros(first + 20, bool)
        at = first + 3                                   # (three blocks hold the prefix)
        for s in range(S):
            n = -(-seen[s] // B)
            table[s, :n] = range(at, at + n)
            at += n
        free[at:at + int(held.sum())] = True
        t = rbkv.StepTables(cfg, S, max_blocks, T)
        t.build(i32(seen), i32(n_new), block_table=i32(table), free=i32(free_words(free)))
        t.append(kn, vn, kc, vc)
        outs.append(t.attention(q, kc, vc, prefix_table=i32(range(first, first + 3)),
                                prefix_len=P).cpu())
        t.device_status()
        del kc, vc
    assert torch.isfinite(outs[0]).all() and torch.equal(*outs)


def test_tensors_at_sixteen_byte_addresses(rbkv):
    """Inputs and outputs that begin 16 bytes into their storage."""
    def shifted(x):
        n = 16 // x.element_size()
        y = torch.empty(x.numel() + n, dtype=x.dtype, device="cuda")[n:].view(x.shape)
        assert y.data_ptr() % 32 == 16
        return y.copy_(x)

    for shape in ((32, 8, 128, 64, "bf16"), (8, 2, 64, 16, "f32")):
        t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 333, *MIXED)
        o = t.attention(q.cuda(), kd, vd, prefix_table=i32(ids), prefix_len=333)
        p = t.attention(shifted(q), shifted(kd), shifted(vd), prefix_table=i32(ids),
                        prefix_len=333, o=shifted(torch.zeros_like(q)))
        t.device_status()
        assert torch.equal(o[:rows], p[:rows])


def test_the_longest_sequence(rbkv):
    """2^30 tokens are the limit of a sequence (256-token blocks)."""
    B, n = 256, 1 << 22
    t = rbkv.StepTables(_cfg(rbkv, block=B, blocks=n), 2, n, 4)
    t.block_table.copy_(torch.arange(n, dtype=torch.int32, device="cuda").expand(2, n))
    t.free.zero_()
    t.build(i32([(1 << 30) - 1, 7]), i32([1, 2]))
    assert t.ctx.tolist() == [1 << 30, 9] and t.slot.tolist() == [(1 << 30) - 1, 7, 8, -1]
    t.device_status()
    t.build(t.ctx, i32([1, 0]))
    assert t.q_start.tolist() == [0, 0, 0] and t.ctx.tolist() == [1 << 30, 9]
    with pytest.raises(rbkv.RbkvError) as e:
        t.device_status()
    assert e.value.status == WORKSPACE


def test_bad_prefix_ids_are_reported(rbkv):
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, 32, 8, 128, 64, "bf16", 200, *MIXED)
    for bad in (-1, 10 ** 6):
        wrong = i32(ids)
        wrong[1] = bad
        t.attention(q.cuda(), kd, vd, prefix_table=wrong, prefix_len=200)
        with pytest.raises(rbkv.RbkvError) as e:
            t.device_status()
        assert e.value.status == BOUNDS
    o = t.attention(q.cuda(), kd, vd, prefix_table=i32(ids), prefix_len=200)
    t.device_status()
    ref = reference(want, q, kc, vc, ids, 200)
    assert ((o[:rows].cpu().double() - ref[0]).abs() <= error_bound(ref, 128, "bf16")).all()


def test_binding_refuses_what_does_not_fit(rbkv):
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, 8, 2, 64, 16, "f32", 20, [3], [1])
    qc = q.cuda()
    wide = torch.randn(*q.shape[:2], 128, device="cuda")[..., :64]
    for args, kw in (((qc.half(), kd, vd), {}), ((wide, kd, vd), {}), ((qc[:, :4], kd, vd), {}),
                     ((qc, kd[1:], vd), {}), ((q, kd, vd), {}),
                     ((qc, kd, vd), {"prefix_table": i32(ids).long(), "prefix_len": 20}),
                     ((qc, kd, vd), {"prefix_table": i32(ids)[:1], "prefix_len": 20})):
        with pytest.raises(ValueError):
            t.attention(*args, **kw)
    with pytest.raises(rbkv.RbkvError):
        t.attention(qc, kd, vd, prefix_len=20)           # a prefix without its blocks
    with pytest.raises(rbkv.RbkvError):
        t.attention(qc, kd, vd, o=qc)
    with pytest.raises(ValueError):
        t.build(i32([3, 3]), i32([1]))
    with pytest.raises(ValueError):
        t.append(qc, qc, kd, vd)


def test_a_step_on_another_stream(rbkv):
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, 32, 8, 128, 64, "bf16", 500, *MIXED)
    qc, idc = q.cuda(), i32(ids)
    here = t.attention(qc, kd, vd, prefix_table=idc, prefix_len=500)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    there = t.attention(qc, kd, vd, prefix_table=idc, prefix_len=500, stream=side)
    t.device_status(stream=side)
    assert torch.equal(here, there)


def test_a_captured_loop_follows_the_lengths(rbkv):
    """One graph - build, append, attention - replayed over steps whose lengths
    change on the device only; every step against the reference."""
    rng = np.random.default_rng(3)
    S, B, hq, hkv, D, T, P = 5, 16, 8, 2, 128, 48, 70
    blocks, max_blocks = 120, 20
    cfg = _cfg(rbkv, hq, hkv, D, B, "bf16", blocks)
    t = rbkv.StepTables(cfg, S, max_blocks, T)
    kc = torch.full(cfg.cache_shape(), float("nan"), dtype=torch.bfloat16, device="cuda")
    vc = kc.clone()
    # the prefix: a step of one sequence whose blocks then stay taken
    pre_k, pre_v = (torch.randn(P, hkv, D).bfloat16().cuda() for _ in range(2))
    first = rbkv.StepTables(cfg, 1, max_blocks, P)
    first.build(i32([0]), i32([P]))
    first.append(pre_k, pre_v, kc, vc)
    ids = first.block_table[0, :-(-P // B)].clone()
    t.free.copy_(first.free)
    q, k, v = (torch.zeros(T, h, D, dtype=torch.bfloat16, device="cuda") for h in (hq, hkv, hkv))
    o = torch.zeros_like(q)
    n_new = torch.zeros(S, dtype=torch.int32, device="cuda")
    ws = torch.empty(max(256, t.workspace_bytes(P)), dtype=torch.uint8, device="cuda")

    def step():
        t.build(t.ctx, n_new)
        t.append(k, v, kc, vc)
        t.attention(q, kc, vc, prefix_table=ids, prefix_len=P, o=o, workspace=ws)

    step()                                   # an empty step, outside the capture
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    ctx = np.zeros(S, np.int64)
    table, free = np.full((S, max_blocks), -1), [False] * len(ids) + [True] * (blocks - len(ids))
    for i in range(12):
        n = rng.choice([0, 1, 1, 9], S) if i else np.array([20, 3, 0, 1, 24])
        for x in (q, k, v):
            x.copy_(torch.randn(x.shape).bfloat16())
        n_new.copy_(i32(n))
        graph.replay()
        torch.cuda.synchronize()
        want = oracle.step.build(ctx, n, table, free, B, T)
        _equal(t, want)
        ctx, table, free = want.ctx, want.table, want.free
        clean = [torch.nan_to_num(x.cpu().float(), 0.0) for x in (kc, vc)]
        ref = reference(want, q.cpu(), *clean, ids.cpu().numpy(), P)
        err = (o.cpu()[:int(n.sum())].double() - ref[0]).abs()
        assert (err <= error_bound(ref, D, "bf16")).all()
    t.device_status()


def test_two_graphs_with_workspaces_of_their_own(rbkv):
    """Two captured steps replayed at once on two streams."""
    runs = []
    for seed in (1, 2):
        t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, 32, 8, 128, 64, "bf16", 600 + seed,
                                                      *MIXED, seed=seed)
        ws = torch.empty(max(256, t.workspace_bytes(600 + seed)), dtype=torch.uint8, device="cuda")
        qc, idc, o = q.cuda(), i32(ids), torch.zeros_like(q).cuda()
        graph = torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph):
            t.attention(qc, kd, vd, prefix_table=idc, prefix_len=600 + seed, o=o, workspace=ws)
        runs.append((graph, torch.cuda.Stream(), o, (t, qc, kd, vd, idc, ws),
                     reference(want, q, kc, vc, ids, 600 + seed), rows))
    for _ in range(20):
        for graph, side, *_ in runs:
            with torch.cuda.stream(side):
                graph.replay()
    torch.cuda.synchronize()
    for _, _, o, keep, ref, rows in runs:
        keep[0].device_status()
        assert ((o[:rows].cpu().double() - ref[0]).abs() <= error_bound(ref, 128, "bf16")).all()


def test_a_decoder_layer_on_a_step(rbkv):
    """The library's decoder layer around a device-built step: the layer's own
    products, and append + attention on the step's tables."""
    from ragged_blocked_kv_gb300.layer import DecoderLayer, random_weights
    hidden, hq, hkv, D, ffn, B, P = 512, 8, 2, 128, 512, 64, 150
    layer = DecoderLayer(rbkv, random_weights(hidden, hq, hkv, D, ffn, seed=4), hq, hkv, D)
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, hq, hkv, D, B, "bf16", P, [70, 0, 9],
                                                  [1, 30, 1])
    x = torch.randn(t.max_tokens, hidden).bfloat16().cuda()
    out, buf, idc = torch.empty_like(x), layer.buffers(t.max_tokens), i32(ids)

    def attend(q, k, v, o):
        t.append(k, v, kd, vd)
        t.attention(q, kd, vd, prefix_table=idc, prefix_len=P, o=o)

    layer.forward_into(x, out, buf, attend, t.max_tokens)
    t.device_status()
    # the attention step's own inputs, as the layer made them
    kn, vn = buf["k"].cpu(), buf["v"].cpu()
    for r in range(rows):
        b, off = divmod(int(want.slot[r]), B)
        kc[b, :, off], vc[b, :, off] = kn[r], vn[r]
    ref = reference(want, buf["q"].cpu(), kc, vc, ids, P)
    err = (buf["o"].cpu()[:rows].double() - ref[0]).abs()
    assert (err <= error_bound(ref, D, "bf16")).all()
    assert torch.isfinite(out).all()
