"""Table builds on a cluster of CTAs: more sequences than a CTA keeps on chip,
refusals found by one CTA of several, the largest pool."""
import numpy as np
import pytest
import torch

import oracle
from step_harness import free_words, i32, random_batch
from test_gpu_step import INVALID, NO_BLOCKS, WORKSPACE, _cfg, _check, _equal

pytestmark = pytest.mark.gpu


def _batch(S, block, longest, new, seed, spare):
    rng = np.random.default_rng(seed)
    seen = rng.integers(0, longest + 1, S)
    n_new = rng.choice(new, S)
    held, need = -(-seen // block), -(-(seen + n_new) // block)
    max_blocks = int(need.max()) + 1
    blocks = int(need.sum()) + spare
    return (seen, n_new, max_blocks, blocks, *random_batch(rng, seen, block, max_blocks,
                                                           blocks)[:2])


def _build(rbkv, t, seen, n_new, table, free, in_place):
    if in_place:
        t.block_table.copy_(i32(table))
        t.free.copy_(i32(free_words(free)))
        t.ctx.copy_(i32(seen))
        t.build(t.ctx, i32(n_new))
    else:
        t.build(i32(seen), i32(n_new), block_table=i32(table), free=i32(free_words(free)))


@pytest.mark.parametrize("S,in_place", [(16384, False), (16385, True), (16385, False),
                                        (20011, True)])
def test_more_sequences_than_fit_on_chip(rbkv, S, in_place):
    """(2048 to a CTA): ragged and idle sequences, two steps and a release."""
    B = 8
    seen, n_new, max_blocks, blocks, table, free = _batch(S, B, 6, [0, 0, 0, 1, 1, 2, 11], S, 900)
    T = int(n_new.sum()) + 3 * S + 5
    t = rbkv.StepTables(_cfg(rbkv, block=B, blocks=blocks + 1000), S, max_blocks + 2, T)
    table = np.concatenate([table, np.full((S, 2), -1)], 1)
    free = np.concatenate([free, np.ones(1000, bool)])
    want = oracle.step.build(seen, n_new, table, free.tolist(), B, T)
    assert want.status == 0
    _build(rbkv, t, seen, n_new, table, free, in_place)
    _equal(t, want)
    more = np.zeros(S, int)
    more[::37] = 3
    again = oracle.step.build(want.ctx, more, want.table, want.free, B, T)
    assert again.status == 0
    t.build(t.ctx, i32(more))
    _equal(t, again)
    done = np.arange(S) % 3 == 0
    t.release(i32(done))
    left = np.array(again.free)
    for s in np.flatnonzero(done):
        left[again.table[s, :-(-int(again.ctx[s]) // B)]] = True
    assert np.array_equal(t.free.cpu().numpy(), free_words(left))
    assert np.array_equal(t.ctx.cpu().numpy(), np.where(done, 0, again.ctx))
    t.device_status()


def test_attention_of_more_sequences_than_fit_on_chip(rbkv):
    rng = np.random.default_rng(12)
    n_new = np.where(rng.random(16500) < 0.05, 1, 0)
    n_new[[3, 9000, 16499]] = [40, 17, 70]
    _check(rbkv, 4, 1, 128, 16, "bf16", 130, rng.integers(0, 20, 16500), n_new, pad=5)


@pytest.mark.parametrize("fault,status,at", [
    ("seen", INVALID, 0), ("n_new", INVALID, 1600), ("table", WORKSPACE, 2999),
    ("longest", WORKSPACE, 1600), ("rows", WORKSPACE, 0), ("blocks", NO_BLOCKS, 0)])
@pytest.mark.parametrize("in_place", [True, False])
def test_refusals_on_a_cluster(rbkv, fault, status, at, in_place):
    """One sequence of 3000, in the first, a middle and the last CTA, makes the
    step one that does not fit: it is empty, and everything is as it was."""
    S, B = 3000, 8
    seen, n_new, max_blocks, blocks, table, free = _batch(S, B, 20, [0, 1, 1, 9], 5, 64)
    T = int(n_new.sum()) + 200
    if fault == "seen":
        seen[at] = -4
    elif fault == "n_new":
        n_new[at] = -1
    elif fault == "table":
        n_new[at] = 150                                  # one row more than its table holds
    elif fault == "longest":
        n_new[at] = 2 ** 31 - 1
    elif fault == "rows":
        T = int(n_new.sum()) - 1
    elif fault == "blocks":
        short = int((-(-(seen + n_new) // B) - -(-seen // B)).sum()) - 1
        free[np.flatnonzero(free)[short:]] = False
    assert fault != "table" or -(-(seen[at] + 150) // B) > max_blocks
    t = rbkv.StepTables(_cfg(rbkv, block=B, blocks=blocks), S, max_blocks, T)
    _build(rbkv, t, seen, n_new, table, free, in_place)
    assert not t.q_start.any() and np.array_equal(t.ctx.cpu().numpy(), seen)
    assert np.array_equal(t.block_table.cpu().numpy(), table)
    assert np.array_equal(t.free.cpu().numpy(), free_words(free))
    assert (t.position == -1).all() and (t.slot == -1).all()
    with pytest.raises(rbkv.RbkvError) as e:
        t.device_status()
    assert e.value.status == status


@pytest.mark.parametrize("blocks", [2 ** 31 - 1, 2 ** 31 - 32, 2 ** 31 - 31])
def test_the_largest_pools(rbkv, blocks):
    """Blocks of one token, as many as a slot can number: the last ones are taken."""
    t = rbkv.StepTables(_cfg(rbkv, block=1, blocks=blocks), 2, 4, 8)
    t.free.zero_()
    t.free[-1] = 1 << ((blocks - 1) % 32) if (blocks - 1) % 32 < 31 else -2 ** 31
    t.free[-2] = 5
    first = (t.free.numel() - 2) * 32
    t.build(i32([0, 0]), i32([1, 2]))
    t.device_status()
    assert t.block_table[:, :2].tolist() == [[first, -1], [first + 2, blocks - 1]]
    assert t.slot.tolist() == [first, first + 2, blocks - 1, -1, -1, -1, -1, -1]
    assert not t.free.any()
    t.release(i32([0, 1]))
    t.device_status()
    assert t.free[-2].item() == 4 and t.free[-1].item() != 0
