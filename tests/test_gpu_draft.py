"""Drafted tokens: the trees' plans, attention over them, acceptance and the move of the
kept rows against the oracle; calls out of order; a captured drafting loop."""
import numpy as np
import pytest
import torch

import oracle
from draft_harness import draft_reference, random_tree, random_trees, rotary_bound
from step_harness import error_bound, free_words, i32, random_batch
from test_gpu_step import BOUNDS, INVALID, _case, _cfg

pytestmark = pytest.mark.gpu
D = oracle.draft


def _status(rbkv, t):
    with pytest.raises(rbkv.RbkvError) as e:
        t.device_status()
    t.device_status()                                     # reading cleared it
    return e.value.status


def _built(rbkv, seen, n_new, block=16, pad=0, seed=0, spare=3, cfg=(), dtype="f32"):
    rng = np.random.default_rng(seed)
    seen, n_new = np.asarray(seen), np.asarray(n_new)
    most = int((-(-(seen + n_new) // block)).max()) + 1
    blocks = int((-(-(seen + n_new) // block)).sum()) + spare
    table, free, _ = random_batch(rng, seen, block, most, blocks)
    T = max(1, int(n_new.sum()) + pad)
    want = oracle.step.build(seen, n_new, table, free, block, T)
    assert want.status == 0
    t = rbkv.StepTables(_cfg(rbkv, *cfg, block=block, dtype=dtype, blocks=blocks), len(seen), most, T)
    t.build(i32(seen), i32(n_new), block_table=i32(table), free=i32(free_words(free)))
    return t, want, rng


# ---- plans -----------------------------------------------------------------------
BATCHES = [([0], [1]), ([7], [128]), ([3, 0, 9], [0, 0, 0]), ([5, 0, 12, 1, 90], [31, 32, 33, 0, 64]),
           ([0, 40, 1, 700], [127, 129, 500, 1]), ([20] * 200, [8] * 200),
           (list(range(300)), [i % 7 for i in range(300)])]


@pytest.mark.parametrize("seen,n_new", BATCHES, ids=lambda x: str(len(x)))
@pytest.mark.parametrize("pad", [0, 700])
def test_plan_against_oracle(rbkv, seen, n_new, pad):
    t, want, rng = _built(rbkv, seen, n_new, pad=pad)
    d = rbkv.StepDraft(t)
    for _ in range(2):
        parent = random_trees(rng, n_new, t.max_tokens)
        d.place.fill_(77)
        d.ancestors.fill_(77)
        d.plan(i32(parent))
        plan = D.plan(want, parent, t.max_tokens)
        assert plan.good
        assert np.array_equal(d.place.cpu().numpy(), plan.place)
        assert np.array_equal(d.ancestors.cpu().numpy(), plan.ancestors)
        t.device_status()


@pytest.mark.parametrize("bad", [
    {0: 0}, {0: -2}, {3: 3}, {3: 2 ** 31 - 1}, {3: -2 ** 31}, {5: 6}, {127: 127}, {127: 128}])
def test_bad_trees_are_chains(rbkv, bad):
    t, want, rng = _built(rbkv, [4, 9, 2], [128, 5, 130], pad=2)
    parent = random_trees(rng, [128, 5, 130], t.max_tokens)
    for i, p in bad.items():
        parent[i] = p
    d = rbkv.StepDraft(t).plan(i32(parent))
    plan = D.plan(want, parent, t.max_tokens)
    assert not plan.good and np.array_equal(d.place.cpu().numpy(), plan.place)
    assert np.array_equal(d.ancestors.cpu().numpy(), plan.ancestors)
    assert _status(rbkv, t) == INVALID
    # a run that is too long for a tree has to be a chain
    parent = random_trees(rng, [128, 5, 130], t.max_tokens)
    parent[133 + 77] = 20
    d.plan(i32(parent))
    assert np.array_equal(d.place.cpu().numpy(), D.plan(want, parent, t.max_tokens).place)
    assert _status(rbkv, t) == INVALID


# ---- attention -------------------------------------------------------------------
TREES = ([0, 0, 5, 63, 64, 200, 17, 0, 31, 130, 1000], [1, 40, 2, 16, 128, 5, 0, 3, 33, 7, 60])
SMALL = ([300, 2, 0], [2, 1, 1])
LONG = ([70, 3, 500], [400, 100, 4])

SHAPES = [(8, 2, 64, 16, "f32"), (4, 4, 32, 5, "f32"), (3, 1, 256, 16, "f32"),
          (8, 2, 64, 16, "bf16"), (6, 2, 96, 24, "bf16"), (32, 32, 128, 64, "bf16"),
          (32, 8, 128, 64, "bf16"), (16, 2, 128, 16, "bf16"), (10, 2, 128, 32, "bf16"),
          (16, 1, 128, 128, "bf16"), (7, 1, 128, 256, "bf16"), (8, 4, 128, 8, "bf16"),
          (64, 1, 128, 64, "bf16")]


def _attend(rbkv, shape, prefix, batch, pad=3, seed=0, parent=None, poison=None, fill=None):
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, prefix, *batch, pad=pad, seed=seed,
                                                  fill=fill)
    rng = np.random.default_rng(seed + 1)
    if parent is None:
        parent = random_trees(rng, batch[1], t.max_tokens)
    if poison is not None:
        poison(want, parent, kc, vc)
        kd, vd = kc.cuda(), vc.cuda()
    d = rbkv.StepDraft(t).plan(i32(parent))
    o = torch.full(q.shape, 7.0, dtype=q.dtype, device="cuda")
    t.attention(q.cuda(), kd, vd, prefix_table=i32(ids) if prefix else None, prefix_len=prefix,
                o=o, draft=d)
    t.device_status()
    o = o.cpu()
    assert (o[rows:] == 7.0).all()
    return t, d, want, parent, q, kc, vc, ids, rows, o


def _check(want, parent, q, kc, vc, ids, prefix, rows, o, shape):
    ref = draft_reference(want, parent, q, kc, vc, ids, prefix)
    err = (o[:rows].double() - ref[0]).abs()
    assert (err <= error_bound(ref, shape[2], shape[4])).all(), float(err.max())


@pytest.mark.parametrize("shape", SHAPES, ids=str)
@pytest.mark.parametrize("prefix", [0, 1, 700])
@pytest.mark.parametrize("batch", [TREES, SMALL, LONG], ids=["trees", "small", "long"])
def test_attention_against_reference(rbkv, shape, prefix, batch):
    t, d, want, parent, q, kc, vc, ids, rows, o = _attend(rbkv, shape, prefix, batch)
    _check(want, parent, q, kc, vc, ids, prefix, rows, o, shape)


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (8, 8, 128, 16, "bf16"),
                                   (8, 2, 64, 16, "f32")], ids=str)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128])
@pytest.mark.parametrize("seen", [0, 1, 15, 100, 127, 128])
def test_sizes_and_alignments_of_one_tree(rbkv, shape, n, seen):
    rng = np.random.default_rng(n * 1000 + seen)
    parent = np.array(random_tree(rng, n) + [0, 0])
    t, d, want, parent, q, kc, vc, ids, rows, o = _attend(rbkv, shape, 0, ([seen], [n]), pad=2,
                                                          seed=n + seen, parent=parent)
    _check(want, parent, q, kc, vc, ids, 0, rows, o, shape)


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (8, 2, 64, 16, "f32"),
                                   (16, 16, 128, 32, "bf16")], ids=str)
def test_roots_alone(rbkv, shape):
    """Every token a root: it sees the cached keys and itself, with none cached itself
    alone, so its output is its value."""
    n = [5, 100, 1]
    t, d, want, parent, q, kc, vc, ids, rows, o = _attend(rbkv, shape, 0, ([0, 0, 0], n),
                                                          parent=np.full(109, -1))
    g = shape[0] // shape[1]
    for r in range(rows):
        b, off = divmod(int(want.slot[r]), shape[3])
        assert torch.equal(o[r], vc[b, :, off].repeat_interleave(g, 0))


@pytest.mark.parametrize("shape", SHAPES[:1] + SHAPES[3:4] + SHAPES[5:8] + SHAPES[11:12], ids=str)
@pytest.mark.parametrize("prefix", [0, 300])
@pytest.mark.parametrize("value", [float("inf"), float("nan"), "lowest"])
def test_what_others_drafted_does_not_reach_a_token(rbkv, shape, prefix, value):
    """Keys and values that are not finite, at tokens that most rows do not follow, and in
    slots that no token has written."""
    if value == "lowest":
        value = torch.finfo(torch.bfloat16 if shape[4] == "bf16" else torch.float32).min
    starts = np.concatenate([[0], np.cumsum(TREES[1])])
    pokes = [(1, 25), (4, 90), (8, 20), (9, 4), (10, 40), (3, 9), (2, 1)]

    def poison(want, parent, kc, vc):
        for s, i in pokes:
            b, off = divmod(int(want.slot[starts[s] + i]), shape[3])
            kc[b, :, off], vc[b, :, off] = value, value

    parent = np.concatenate([[-1 if i == 0 else (i - 1) // 2 for i in range(n)]
                             for n in TREES[1]] + [[0, 0, 0]]).astype(np.int64)
    t, d, want, parent, q, kc, vc, ids, rows, o = _attend(rbkv, shape, prefix, TREES, seed=4,
                                                          parent=parent, poison=poison, fill=value)
    hit = torch.zeros(rows, dtype=torch.bool)
    for s, i in pokes:
        p, _ = D.parents_of(want, parent, s)
        for j in range(len(p)):
            hit[starts[s] + j] |= i in D.way_up(p, j)
    kc, vc = (torch.nan_to_num(x.float(), 0, 0, 0) for x in (kc, vc))
    kc, vc = (torch.where(x.abs() > 1e30, 0.0, x) for x in (kc, vc))
    ref = draft_reference(want, parent, q, kc, vc, ids, prefix)
    err = (o[:rows].double() - ref[0]).abs()
    assert (err[~hit] <= error_bound(ref, shape[2], shape[4])[~hit]).all()
    assert hit.sum() >= len(pokes) and (~hit).sum() > rows // 2


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (8, 8, 128, 16, "bf16"),
                                   (8, 2, 64, 16, "bf16"), (8, 2, 64, 16, "f32")], ids=str)
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_values_reach_the_rows_that_follow_them(rbkv, shape, value):
    """A value that is not finite reaches every row that follows its token, even behind a
    weight that underflows to 0."""
    batch = ([70, 3, 500, 9], [128, 12, 2, 3])
    starts = np.concatenate([[0], np.cumsum(batch[1])])
    pokes = [(0, 40), (1, 5), (2, 1), (3, 0)]
    parent = np.concatenate([[-1 if i == 0 else (i - 1) // 3 for i in range(n)]
                             for n in batch[1]] + [[0, 0, 0]]).astype(np.int64)

    def change(q, kn, vn):
        q.copy_(1 + q.abs())
        for s, i in pokes:
            kn[starts[s] + i] = -1600 / shape[2] ** 0.5
            vn[starts[s] + i, :, 7] = value

    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 0, *batch, pad=3, seed=8,
                                                  change=change)
    d = rbkv.StepDraft(t).plan(i32(parent))
    o = t.attention(q.cuda(), kd, vd, draft=d).cpu()[:rows].double()
    hit = torch.zeros(rows, shape[0], shape[2], dtype=torch.bool)
    for s, i in pokes:
        p, _ = D.parents_of(want, parent, s)
        for j in range(len(p)):
            if i in D.way_up(p, j):
                hit[starts[s] + j, :, 7] = True
    assert not torch.isfinite(o[hit]).any()
    vc = torch.nan_to_num(vc.float(), 0, 0, 0)
    ref = draft_reference(want, parent, q, kc, vc, ids, 0)
    err = (o - ref[0]).abs()
    assert (err[~hit] <= error_bound(ref, shape[2], shape[4])[~hit]).all()


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (8, 4, 128, 8, "bf16"),
                                   (8, 2, 64, 16, "f32")], ids=str)
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_bad_block_ids_are_left_out(rbkv, shape, bad):
    """The first block of a sequence, and the last (which holds drafted tokens)."""
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 0, *TREES, pad=1)
    parent = random_trees(np.random.default_rng(2), TREES[1], t.max_tokens)
    d = rbkv.StepDraft(t).plan(i32(parent))
    B = shape[3]
    gone = [(5, 0), (10, 1059 // B), (4, 191 // B)]
    table = want.table.copy()
    for s, c in gone:
        table[s, c] = bad
    t.block_table.copy_(i32(table))
    o = t.attention(q.cuda(), kd, vd, draft=d).cpu()[:rows].double()
    assert _status(rbkv, t) == BOUNDS
    assert torch.isfinite(o).all()
    same = torch.ones(rows, dtype=torch.bool)
    for s, c in gone:
        same[int(want.q_start[s]):int(want.q_start[s + 1])] = False
    ref = draft_reference(want, parent, q, kc, vc, ids, 0)
    err = (o - ref[0]).abs()
    assert (err[same] <= error_bound(ref, shape[2], shape[4])[same]).all()
    # sequence 5: by hand over the keys that are left
    p, _ = D.parents_of(want, parent, 5)
    q0, seen, g = int(want.q_start[5]), TREES[0][5], shape[0] // shape[1]
    for i in range(len(p)):
        at = [x for x in list(range(seen)) + [seen + j for j in D.way_up(p, i)] if x >= B]
        slots = [int(want.table[5, x // B]) * B + x % B for x in at]
        k, v = (torch.stack([c[s // B, :, s % B] for s in slots]).double() for c in (kc, vc))
        x = torch.einsum("hgd,khd->hgk", q[q0 + i].double().view(-1, g, shape[2]), k)
        w = torch.softmax(x / shape[2] ** 0.5, -1)
        exact = torch.einsum("hgk,khd->hgd", w, v).reshape(shape[0], shape[2])
        size = torch.einsum("hgk,khd->hgd", w, v.abs()).reshape(shape[0], shape[2])
        assert ((o[q0 + i] - exact).abs() <= 2.0 ** -6 * size + 1e-4).all()


def test_calls_out_of_order(rbkv):
    """Nothing is done with trees of another step, or a path that has not been taken."""
    shape = (8, 2, 128, 16, "bf16")
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 0, [5, 40], [6, 4])
    d = rbkv.StepDraft(t)
    qd, o = q.cuda(), torch.full_like(q, 7.0, device="cuda")
    tok = torch.zeros(t.max_tokens, dtype=torch.int32, device="cuda")
    parent = i32(random_trees(np.random.default_rng(0), [6, 4], t.max_tokens))
    ctx, free = t.ctx.clone(), t.free.clone()

    def refused(call):
        call()
        assert _status(rbkv, t) == INVALID
        assert (o == 7.0).all() and torch.equal(t.ctx, ctx) and torch.equal(t.free, free)
        assert torch.equal(kd.cpu(), kc) and (d.path == -1).all() and not d.accepted.any()

    refused(lambda: t.attention(qd, kd, vd, o=o, draft=d))
    refused(lambda: d.accept(tok, tok))
    refused(lambda: d.compact(kd, vd))
    d.plan(parent)
    refused(lambda: d.compact(kd, vd))
    t.attention(qd, kd, vd, o=o, draft=d)
    t.device_status()
    t.build(t.ctx, i32([0, 0]))                          # the trees are the last step's
    o.fill_(7.0)
    t.attention(qd, kd, vd, o=o, draft=d)                # (no rows: nothing to report)
    t.device_status()
    t.build(t.ctx, i32([1, 2]))
    ctx, free = t.ctx.clone(), t.free.clone()
    refused(lambda: t.attention(qd, kd, vd, o=o, draft=d))
    refused(lambda: d.accept(tok, tok))
    d.plan(i32([-1, -1, 0] + [0] * (t.max_tokens - 3)))
    t.device_status()
    late = rbkv.StepDraft(t)                             # (planned by another: not by this one)
    refused(lambda: t.attention(qd, kd, vd, o=o, draft=late))
    refused(lambda: late.accept(tok, tok))
    # f32 shapes, on the CUDA cores
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, 8, 2, 64, 16, "f32", 0, [5, 40], [6, 4])
    d, o = rbkv.StepDraft(t), torch.full_like(q, 7.0, device="cuda")
    t.attention(q.cuda(), kd, vd, o=o, draft=d)
    assert _status(rbkv, t) == INVALID and (o == 7.0).all()


WIDE = ([1000, 30, 2000, 70, 0, 3000, 128, 640], [128, 100, 64, 33, 500, 65, 97, 1])


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (16, 1, 128, 16, "bf16"),
                                   (10, 2, 128, 32, "bf16"), (64, 1, 128, 128, "bf16"),
                                   (7, 7, 128, 8, "bf16")], ids=str)
@pytest.mark.parametrize("prefix", [0, 900])
@pytest.mark.parametrize("batch", [WIDE, ([5000], [128]), ([0, 9000], [128, 90]),
                                   ([300] * 40, [70] * 40)], ids=["wide", "one", "two", "many"])
def test_several_query_tiles_per_sequence(rbkv, shape, prefix, batch):
    """Odd and even numbers of query tiles, of different lengths, over few and many keys."""
    t, d, want, parent, q, kc, vc, ids, rows, o = _attend(rbkv, shape, prefix, batch, seed=11)
    _check(want, parent, q, kc, vc, ids, prefix, rows, o, shape)


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (16, 1, 128, 16, "bf16"),
                                   (9, 9, 128, 32, "bf16")], ids=str)
@pytest.mark.parametrize("prefix", [0, 300])
def test_long_chains_in_pairs(rbkv, shape, prefix):
    """Prompt chunks behind many keys beside trees: pairs whose first tile has fewer keys,
    the last one not whole."""
    batch = ([2000, 0, 5000, 70, 1500], [700, 1300, 128, 300, 333])
    t, d, want, parent, q, kc, vc, ids, rows, o = _attend(rbkv, shape, prefix, batch, seed=12)
    _check(want, parent, q, kc, vc, ids, prefix, rows, o, shape)


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (16, 1, 128, 16, "bf16"),
                                   (9, 9, 128, 32, "bf16")], ids=str)
@pytest.mark.parametrize("prefix", [0, 900])
@pytest.mark.parametrize("value", [float("inf"), float("nan")])
def test_pairs_with_values_that_are_not_finite(rbkv, shape, prefix, value):
    """As the two tests above, where query tiles are walked in pairs: what a token does not
    follow does not reach it, what it follows does."""
    starts = np.concatenate([[0], np.cumsum(WIDE[1])])
    pokes = [(0, 90), (1, 99), (2, 40), (4, 300), (5, 3), (7, 0)]

    def poison(want, parent, kc, vc):
        for s, i in pokes:
            b, off = divmod(int(want.slot[starts[s] + i]), shape[3])
            vc[b, :, off, 5] = value

    parent = np.concatenate([D.chain(n) if n > 128 else
                             [-1 if i == 0 else (i - 1) // 2 for i in range(n)]
                             for n in WIDE[1]] + [[0, 0, 0]]).astype(np.int64)
    t, d, want, parent, q, kc, vc, ids, rows, o = _attend(rbkv, shape, prefix, WIDE, seed=13,
                                                          parent=parent, poison=poison, fill=value)
    hit = torch.zeros(o[:rows].shape, dtype=torch.bool)
    for s, i in pokes:
        p, _ = D.parents_of(want, parent, s)
        for j in range(len(p)):
            if i in D.way_up(p, j):
                hit[starts[s] + j, :, 5] = True
    kc, vc = (torch.nan_to_num(x.float(), 0, 0, 0) for x in (kc, vc))
    ref = draft_reference(want, parent, q, kc, vc, ids, prefix)
    err = (o[:rows].double() - ref[0]).abs()
    assert (err[~hit] <= error_bound(ref, shape[2], shape[4])[~hit]).all()
    assert not torch.isfinite(o[:rows][hit]).any()


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (16, 1, 128, 16, "bf16")], ids=str)
def test_pairs_with_bad_block_ids(rbkv, shape):
    """The first block of the first sequence (a call's first tile) and the last of others."""
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 0, *WIDE, pad=1)
    parent = random_trees(np.random.default_rng(2), WIDE[1], t.max_tokens)
    d = rbkv.StepDraft(t).plan(i32(parent))
    gone = [(0, 0), (2, 2063 // shape[3]), (5, 100 // shape[3])]
    table = want.table.copy()
    for s, c in gone:
        table[s, c] = 10 ** 6
    t.block_table.copy_(i32(table))
    o = t.attention(q.cuda(), kd, vd, draft=d).cpu()[:rows].double()
    assert _status(rbkv, t) == BOUNDS
    own = torch.zeros(rows, dtype=torch.bool)
    for s, c in gone:
        own[int(want.q_start[s]):int(want.q_start[s + 1])] = True
    ref = draft_reference(want, parent, q, kc, vc, ids, 0)
    err = (o - ref[0]).abs()
    assert (err[~own] <= error_bound(ref, shape[2], shape[4])[~own]).all()
    assert torch.isfinite(o).all() and (err[own] > 0).any()


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (8, 2, 64, 16, "f32")], ids=str)
def test_tensors_on_16_byte_addresses(rbkv, shape):
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 0, *TREES, pad=1)
    parent = random_trees(np.random.default_rng(3), TREES[1], t.max_tokens)
    n = 16 // q.element_size()

    def off(x):
        y = torch.zeros(x.numel() + n, dtype=x.dtype, device="cuda")[n:].view(x.shape)
        return y.copy_(x)

    qd, o, kd, vd = off(q), off(torch.zeros_like(q)), off(kc), off(vc)
    assert qd.data_ptr() % 32 == 16
    d = rbkv.StepDraft(t).plan(i32(parent))
    t.attention(qd, kd, vd, o=o, draft=d)
    t.device_status()
    _check(want, parent, q, kc, vc, ids, 0, rows, o.cpu(), shape)


# ---- acceptance ------------------------------------------------------------------
@pytest.mark.parametrize("seen,n_new", BATCHES + [([60, 5, 31], [90, 300, 20])],
                         ids=lambda x: str(len(x)))
@pytest.mark.parametrize("given", [False, True])
@pytest.mark.parametrize("words", [1, 2, 50])
def test_accept_and_compact_against_oracle(rbkv, seen, n_new, given, words):
    """Few different tokens, so that paths are long and siblings alike."""
    t, want, rng = _built(rbkv, seen, n_new, block=8, pad=4, seed=words, cfg=(8, 2, 128))
    T, S = t.max_tokens, t.num_seqs
    parent = random_trees(rng, n_new, T)
    tokens, chosen = rng.integers(0, words, T), rng.integers(0, words, T)
    first = np.array([rng.integers(1, n + 1) if n else rng.integers(-3, 3) for n in n_new])
    d = rbkv.StepDraft(t).plan(i32(parent))
    gen = torch.Generator().manual_seed(words)
    kc, vc = (torch.randn(t.config.cache_shape(), generator=gen) for _ in range(2))
    kd, vd = kc.cuda(), vc.cuda()
    done = D.accept(want, parent, tokens, chosen, first if given else None, 8)
    d.accept(i32(tokens), i32(chosen), i32(first) if given else None)
    d.compact(kd, vd)
    t.device_status()

    def check():
        assert np.array_equal(d.path.cpu().numpy(), done.path)
        assert d.accepted.tolist() == done.accepted.tolist()
        assert d.next_token.tolist() == done.next_token.tolist()
        assert t.ctx.tolist() == done.ctx.tolist()
        assert np.array_equal(t.free.cpu().numpy(), free_words(done.free))

    check()
    assert np.array_equal(t.block_table.cpu().numpy(), want.table)
    assert np.array_equal(t.slot.cpu().numpy(), want.slot)
    for c, x in ((kc, kd), (vc, vd)):
        D.compact(want, done, c, 8)
        assert torch.equal(c, x.cpu())
    d.accept(i32(tokens), i32(chosen), i32(first) if given else None)      # the same again
    check()
    t.device_status()


def test_thousands_of_sequences(rbkv):
    """Plans, acceptance and move of 5000 sequences; more kept for a plan than a thread holds."""
    S = 5000
    rng = np.random.default_rng(21)
    n_new = rng.integers(0, 9, S)
    n_new[::500] = 100
    t, want, rng = _built(rbkv, rng.integers(0, 90, S), n_new, block=32, seed=3, cfg=(8, 1, 128),
                          dtype="bf16")
    T = t.max_tokens
    parent = random_trees(rng, n_new, T)
    tokens, chosen = rng.integers(0, 2, T), rng.integers(0, 2, T)
    d = rbkv.StepDraft(t).plan(i32(parent))
    plan = D.plan(want, parent, T)
    assert np.array_equal(d.place.cpu().numpy(), plan.place)
    assert np.array_equal(d.ancestors.cpu().numpy(), plan.ancestors)
    caches = [torch.randn(t.config.cache_shape()).to(torch.bfloat16) for _ in range(2)]
    dev = [c.cuda() for c in caches]
    done = D.accept(want, parent, tokens, chosen, None, 32)
    d.accept(i32(tokens), i32(chosen))
    d.compact(*dev)
    t.device_status()
    assert np.array_equal(d.path.cpu().numpy(), done.path)
    assert t.ctx.tolist() == done.ctx.tolist()
    assert np.array_equal(t.free.cpu().numpy(), free_words(done.free))
    for c, x in zip(caches, dev):
        D.compact(want, done, c, 32)
        assert torch.equal(c, x.cpu())
    q = torch.randn(T, 8, 128).to(torch.bfloat16)
    kc, vc = caches
    rows = int(want.q_start[-1])
    o = t.attention(q.cuda(), *dev, draft=d).cpu()
    t.device_status()
    ref = draft_reference(want, parent, q, kc, vc, [], 0)
    err = (o[:rows].double() - ref[0]).abs()
    assert (err <= error_bound(ref, 128, "bf16")).all()


def test_given_out_of_range(rbkv):
    t, want, rng = _built(rbkv, [3, 9, 0], [6, 5, 200])
    parent = random_trees(rng, [6, 5, 200], t.max_tokens)
    tok = np.zeros(t.max_tokens, np.int64)
    d = rbkv.StepDraft(t).plan(i32(parent))
    for given in ([0, 1, 1], [1, 6, 1], [1, 1, 201], [1, 1, -5], [2 ** 31 - 1, -2 ** 31, 1]):
        d.accept(i32(tok), i32(tok + 1), i32(given))
        done = D.accept(want, parent, tok, tok + 1, given, 16)
        assert d.accepted.tolist() == done.accepted.tolist()
        assert np.array_equal(d.path.cpu().numpy(), done.path)
        assert _status(rbkv, t) == INVALID


@pytest.mark.parametrize("shape", [(4, 4, 32, 5, "f32"), (64, 64, 256, 16, "bf16"),
                                   (3, 1, 96, 24, "bf16")], ids=str)
def test_compact_moves_whole_rows(rbkv, shape):
    """Overlapping moves of long paths, every row width."""
    hq, hkv, dim, block, dtype = shape
    n_new = [128, 77, 1, 40]
    t, want, rng = _built(rbkv, [3, 0, 9, 12], n_new, block=block, cfg=(hq, hkv, dim), dtype=dtype)
    parent = np.concatenate([[-1] + [max(0, i - 2) for i in range(1, n)] for n in n_new])
    d = rbkv.StepDraft(t).plan(i32(parent))
    tok = np.zeros(t.max_tokens, np.int64)
    done = D.accept(want, parent, tok, tok, None, block)
    d.accept(i32(tok), i32(tok))
    caches = [torch.randn(t.config.cache_shape()).to(t.config.torch_dtype) for _ in range(2)]
    dev = [c.cuda() for c in caches]
    d.compact(*dev)
    t.device_status()
    for c, x in zip(caches, dev):
        D.compact(want, done, c, block)
        assert torch.equal(c, x.cpu())


def test_compact_past_two_to_the_31(rbkv):
    blocks = 33000                                       # 33000 * 65536 elements
    cfg = rbkv.Config(8, 8, 128, 64, "bf16", blocks)
    t = rbkv.StepTables(cfg, 1, 4, 5)
    t.free.zero_()
    t.free[(blocks - 1) // 32] = 1 << ((blocks - 1) % 32)
    t.build(t.ctx, i32([5]))
    d = rbkv.StepDraft(t).plan(i32([-1, 0, 0, 0, 3]))
    tokens = i32([1, 2, 3, 4, 5])
    d.accept(tokens, i32([4, 0, 0, 5, 9]))
    assert d.path.tolist() == [0, 3, 4, -1, -1] and d.next_token.tolist() == [9]
    kd, vd = (torch.zeros(cfg.cache_shape(), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    kd[-1, :, :5] = torch.arange(1, 6, device="cuda")[:, None].to(torch.bfloat16)
    d.compact(kd, vd)
    t.device_status()
    assert kd[-1, 3, :5, 7].tolist() == [1, 4, 5, 4, 5] and not kd[0].any()


# ---- a drafting loop ---------------------------------------------------------------
@pytest.mark.parametrize("shape", [(16, 4, 128, 16, "bf16"), (8, 2, 64, 8, "f32")], ids=str)
@pytest.mark.parametrize("captured", [False, True])
def test_a_drafting_loop(rbkv, shape, captured):
    """Eight steps of two layers behind a shared prefix: trees, an idle slot, a prompt chunk
    in the first step; every array, cache and output checked after each."""
    hq, hkv, dim, block, dtype = shape
    S, T, P, blocks, most = 4, 60, 3 * block + 1, 80, 16
    cfg = rbkv.Config(*shape, blocks)
    rng = np.random.default_rng(9)
    gen = torch.Generator().manual_seed(9)
    dt = cfg.torch_dtype
    t = rbkv.StepTables(cfg, S, most, T)
    d = rbkv.StepDraft(t)
    rope = rbkv.Rotary(dim, base=100.0)
    ids = np.arange(blocks - 4, blocks)
    free = np.ones(blocks, bool)
    free[ids] = False
    t.free.copy_(i32(free_words(free)))
    layers = [[torch.randn(cfg.cache_shape(), generator=gen).to(dt) for _ in range(2)]
              for _ in range(2)]
    dev = [[c.cuda() for c in pair] for pair in layers]
    n_new, parent, tokens, chosen, given = (torch.zeros(n, dtype=torch.int32, device="cuda")
                                            for n in (S, T, T, T, S))
    rows_in = [[torch.zeros(T, h, dim, dtype=dt, device="cuda") for h in (hq, hkv, hkv)]
               for _ in range(2)]
    q_out = [torch.zeros(T, hq, dim, dtype=dt, device="cuda") for _ in range(2)]
    outs = [torch.zeros_like(q_out[0]) for _ in range(2)]
    ws = torch.empty(max(256, t.workspace_bytes(P)), dtype=torch.uint8, device="cuda")
    idc = i32(ids)

    def step():
        t.build(t.ctx, n_new)
        d.plan(parent)
        for (kc, vc), (q, k, v), qo, o in zip(dev, rows_in, q_out, outs):
            t.append_rotary(rope, q, k, v, kc, vc, q_out=qo, prefix_len=P, draft=d)
            t.attention(qo, kc, vc, prefix_table=idc, prefix_len=P, o=o, workspace=ws, draft=d)
        d.accept(tokens, chosen, given)
        for kc, vc in dev:
            d.compact(kc, vc)

    graph = None
    if captured:
        step()                                            # (an empty step)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    ctx, table = np.zeros(S, np.int64), np.full((S, most), -1)
    moved = 0
    for i in range(8):
        new = rng.integers(1, 12, S)
        new[i % S] = 0
        if i == 0:
            new[2] = 30
        want = oracle.step.build(ctx, new, table, list(free), block, T)
        assert want.status == 0
        rows = int(want.q_start[-1])
        tree = random_trees(rng, new, T)
        first = np.where(new > 0, 1, 0)
        if i == 0:
            tree[want.q_start[2]:want.q_start[3]] = D.chain(30)
            first[2] = 30
        tok, pick = rng.integers(0, 2, T), rng.integers(0, 2, T)
        for a, b in ((n_new, new), (parent, tree), (tokens, tok), (chosen, pick), (given, first)):
            a.copy_(i32(b))
        host = []
        for x in rows_in:
            fresh = [torch.randn(y.shape, generator=gen).to(dt) for y in x]
            for a, b in zip(x, fresh):
                a.copy_(b)
            host.append(fresh)
        graph.replay() if captured else step()
        torch.cuda.synchronize()
        t.device_status()
        plan = D.plan(want, tree, T)
        done = D.accept(want, tree, tok, pick, first, block)
        assert np.array_equal(d.path.cpu().numpy(), done.path)
        assert t.ctx.tolist() == done.ctx.tolist()
        assert np.array_equal(t.free.cpu().numpy(), free_words(done.free))
        moved += int((done.path > np.arange(T)).sum())
        slot = torch.from_numpy(want.slot[:rows].astype(np.int64))
        place = plan.place[:rows] + P
        for (kc, vc), (kd, vd), (q, k, v), qo, o in zip(layers, dev, host, q_out, outs):
            exact = D.rotate(q[:rows].double().numpy(), place, rope.inv_freq, "half")
            bound = rotary_bound(q[:rows].double().numpy(), place, rope.inv_freq, "half", 1.0,
                                 exact, dtype)
            assert (np.abs(qo[:rows].double().cpu().numpy() - exact) <= bound).all()
            # (the keys as the kernel rotated them, from a second call on other caches)
            spare = [torch.zeros_like(kd) for _ in range(2)]
            t.append_rotary(rope, *(x.cuda() for x in (q, k, v)), *spare, prefix_len=P, draft=d)
            mine = spare[0].cpu()[slot // block, :, slot % block]
            exact = D.rotate(k[:rows].double().numpy(), place, rope.inv_freq, "half")
            bound = rotary_bound(k[:rows].double().numpy(), place, rope.inv_freq, "half", 1.0,
                                 exact, dtype)
            assert (np.abs(mine.double().numpy() - exact) <= bound).all()
            kc[slot // block, :, slot % block] = mine
            vc[slot // block, :, slot % block] = v[:rows]
            _check(want, tree, qo.cpu(), kc, vc, ids, P, rows, o.cpu(), shape)
            D.compact(want, done, kc, block)
            D.compact(want, done, vc, block)
            assert torch.equal(kd.cpu(), kc) and torch.equal(vd.cpu(), vc)
        ctx, table = done.ctx, want.table
        for s in range(S):
            table[s, -(-int(ctx[s]) // block):] = -1
        free = np.array(done.free)
    assert moved > 5


def test_two_drafts_on_two_streams(rbkv):
    """Two tables and drafts at once, a workspace each; the cache is shared."""
    shape = (32, 8, 128, 64, "bf16")
    runs = []
    for i in range(2):
        t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 0, *TREES, pad=1, seed=i)
        parent = random_trees(np.random.default_rng(i), TREES[1], t.max_tokens)
        ws = torch.empty(max(256, t.workspace_bytes(0)), dtype=torch.uint8, device="cuda")
        runs.append((t, rbkv.StepDraft(t), i32(parent), q.cuda(), kd, vd,
                     torch.zeros_like(q, device="cuda"), ws, torch.cuda.Stream(),
                     (want, parent, q, kc, vc, ids, rows)))
    torch.cuda.synchronize()
    for _ in range(10):
        for t, d, parent, q, kd, vd, o, ws, side, _ in runs:
            d.plan(parent, stream=side)
            t.attention(q, kd, vd, o=o, workspace=ws, stream=side, draft=d)
    torch.cuda.synchronize()
    for t, d, _, _, _, _, o, _, _, (want, parent, q, kc, vc, ids, rows) in runs:
        t.device_status()
        _check(want, parent, q, kc, vc, ids, 0, rows, o.cpu(), shape)
