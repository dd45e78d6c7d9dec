"""Drafted tokens behind blocks that are not in the pool, and two batches over one cache."""
import math

import numpy as np
import pytest
import torch

import oracle
from draft_harness import draft_reference, random_trees
from step_harness import error_bound, i32
from test_gpu_draft import LONG, TREES, WIDE, _check, _status
from test_gpu_step import BOUNDS, _case

pytestmark = pytest.mark.gpu
D = oracle.draft


def _without(ref, want, parent, q, k_cache, v_cache, gone):
    """`ref` (of draft_reference, no prefix) with the rows of the sequences in `gone` - (sequence,
    column of its table) - taken over the keys that are left; a row that has none is 0."""
    B, H_kv, dim = k_cache.shape[2], k_cache.shape[1], q.shape[2]
    g = q.shape[1] // H_kv
    out, absv, absqk, keys = (x.clone() for x in ref)
    for s in sorted({s for s, _ in gone}):
        a, b = int(want.q_start[s]), int(want.q_start[s + 1])
        n = int(want.ctx[s])
        seen = n - (b - a)
        at = torch.arange(n)
        left = torch.tensor([(s, int(x) // B) not in gone for x in at])
        p, _ = D.parents_of(want, parent, s)
        sees = torch.zeros(b - a, n, dtype=torch.bool)
        sees[:, :seen] = True
        for i in range(b - a):
            sees[i, [seen + j for j in D.way_up(p, i)]] = True
        sees &= left
        ids = torch.from_numpy(want.table[s].astype(np.int64))[at // B]
        k, v = (c[ids, :, at % B].double().permute(1, 0, 2) for c in (k_cache, v_cache))
        qs = q[a:b].double().reshape(b - a, H_kv, g, dim).permute(1, 2, 0, 3)
        x = (qs @ k[:, None].transpose(2, 3) / math.sqrt(dim)).masked_fill(~sees, -math.inf)
        w = torch.nan_to_num(torch.softmax(x, -1), nan=0.0)

        def back(y):
            return y.permute(2, 0, 1, 3).reshape(b - a, H_kv * g, -1)

        out[a:b], absv[a:b] = back(w @ v[:, None]), back(w @ v.abs()[:, None])
        ax = qs.abs() @ k[:, None].abs().transpose(2, 3) / math.sqrt(dim)
        absqk[a:b] = back(ax.masked_fill(~sees, 0.0).amax(-1, keepdim=True))
        keys[a:b, 0, 0] = sees.sum(1).double()
    return out, absv, absqk, keys


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (16, 1, 128, 16, "bf16"),
                                   (8, 4, 128, 8, "bf16"), (8, 2, 64, 16, "f32")], ids=str)
@pytest.mark.parametrize("batch", [TREES, LONG, WIDE, ([300] * 40, [70] * 40)],
                         ids=["trees", "long", "wide", "many"])
@pytest.mark.parametrize("bad", [-1, 10 ** 6])
def test_rows_over_the_keys_that_are_left(rbkv, shape, batch, bad):
    """Each sequence loses its first, a middle or its last block (where drafted tokens lie):
    the keys are left out, not taken for zeros."""
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 0, *batch, pad=1, seed=5)
    parent = random_trees(np.random.default_rng(5), batch[1], t.max_tokens)
    B, table, gone = shape[3], want.table.copy(), set()
    for s, n in enumerate(batch[1]):
        blocks = -(-int(want.ctx[s]) // B)
        if n > 0 and s % 4 < 3:
            gone.add((s, (0, blocks // 2, blocks - 1)[s % 4]))
    for s, c in gone:
        table[s, c] = bad
    d = rbkv.StepDraft(t).plan(i32(parent))
    t.block_table.copy_(i32(table))
    o = t.attention(q.cuda(), kd, vd, draft=d).cpu()[:rows].double()
    assert _status(rbkv, t) == BOUNDS
    full = draft_reference(want, parent, q, kc, vc, ids, 0)
    ref = _without(full, want, parent, q, kc, vc, gone)
    bound = error_bound(ref, shape[2], shape[4])
    err = (o - ref[0]).abs()
    assert (err <= bound).all(), float(err.max())
    # (a row's missing keys change it by more than any rounding, as a rule)
    lost = torch.zeros(rows, dtype=torch.bool)
    for s, _ in gone:
        lost[int(want.q_start[s]):int(want.q_start[s + 1])] = True
    far = ((full[0] - ref[0]).abs() > 2 * bound).flatten(1).any(1)
    assert far[lost].double().mean() > 0.5 and not far[~lost].any()


def test_a_row_with_no_key_left_is_zero(rbkv):
    shape = (32, 8, 128, 64, "bf16")
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 0, [0, 3], [50, 40])
    d = rbkv.StepDraft(t).plan(i32(np.concatenate([D.chain(50), D.chain(40)])))
    t.block_table[0].fill_(-1)
    o = t.attention(q.cuda(), kd, vd, draft=d).cpu()
    assert _status(rbkv, t) == BOUNDS
    assert not o[:50].any() and torch.isfinite(o).all() and o[50:90].any(-1).all()


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (8, 2, 64, 16, "f32")], ids=str)
def test_two_drafts_over_one_cache(rbkv, shape):
    """Two tables of the same blocks, two drafts of other trees, on two streams at once."""
    runs = []
    for i in range(2):
        t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 0, *TREES, pad=1, seed=6)
        parent = random_trees(np.random.default_rng(i), TREES[1], t.max_tokens)
        if i:
            kd, vd = runs[0][4:6]
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
    assert runs[0][4].data_ptr() == runs[1][4].data_ptr()
    for t, d, _, _, _, _, o, _, _, (want, parent, q, kc, vc, ids, rows) in runs:
        t.device_status()
        _check(want, parent, q, kc, vc, ids, 0, rows, o.cpu(), shape)


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (16, 2, 128, 16, "bf16"),
                                   (8, 2, 64, 16, "f32")], ids=str)
@pytest.mark.parametrize("prefix", [0, 700])
def test_the_same_call_gives_the_same_bits(rbkv, shape, prefix):
    """Cuts, spills and their joins go by the lengths alone, not by which CTA is first."""
    batch = ([2000, 0, 5, 63, 64, 5000, 17], [128, 40, 2, 16, 300, 90, 5])
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, prefix, *batch, seed=7)
    d = rbkv.StepDraft(t).plan(i32(random_trees(np.random.default_rng(7), batch[1], t.max_tokens)))
    qd, idc = q.cuda(), i32(ids) if prefix else None
    first = t.attention(qd, kd, vd, prefix_table=idc, prefix_len=prefix, draft=d).cpu()
    for _ in range(20):
        o = t.attention(qd, kd, vd, prefix_table=idc, prefix_len=prefix, draft=d)
        assert torch.equal(o.cpu()[:rows], first[:rows])
    t.device_status()
