"""What an acceptance of drafted tokens keeps, and what it gives back."""
import numpy as np
import pytest
import torch

import oracle
from draft_harness import random_trees
from step_harness import free_words, i32
from test_gpu_draft import _built, _status
from test_gpu_step import INVALID

pytestmark = pytest.mark.gpu
D = oracle.draft


def _kept(t, d, done):
    assert np.array_equal(d.path.cpu().numpy(), done.path)
    assert d.accepted.tolist() == done.accepted.tolist()
    assert d.next_token.tolist() == done.next_token.tolist()
    assert t.ctx.tolist() == done.ctx.tolist()
    assert np.array_equal(t.free.cpu().numpy(), free_words(done.free))


def _built_again(rng, t, done, last, seen, n_new, block):
    """The next step (no longer than the last): tables, no block held twice or held and
    free."""
    n_new = np.array([rng.integers(0, min(n, a + n - int(c)) + 1)
                      for a, n, c in zip(seen, n_new, done.ctx)])
    want = oracle.step.build(done.ctx, n_new, last.table, done.free, block, t.max_tokens)
    assert want.status == 0
    t.build(t.ctx, i32(n_new))
    t.device_status()
    assert t.ctx.tolist() == want.ctx.tolist()
    assert np.array_equal(t.free.cpu().numpy(), free_words(want.free))
    assert np.array_equal(t.slot.cpu().numpy(), want.slot)
    held = [t.block_table[s, :-(-int(c) // block)] for s, c in enumerate(want.ctx)]
    held = torch.cat(held).tolist()
    assert len(held) == len(set(held)) and not any(want.free[b] for b in held)


# ---- a second acceptance -----------------------------------------------------------
KEEP = [([0], [128]), ([60, 5, 31, 0], [90, 300, 20, 0]), ([7, 8, 9, 16], [17, 16, 1, 40]),
        ([20] * 200, [9] * 200)]


@pytest.mark.parametrize("seen,n_new", KEEP, ids=lambda x: str(len(x)))
@pytest.mark.parametrize("block", [1, 8, 64])
def test_another_acceptance_of_the_same_step(rbkv, seen, n_new, block):
    """Short, long and short paths in turn: what is held and what is free goes by the last."""
    t, want, rng = _built(rbkv, seen, n_new, block=block, seed=block)
    T = t.max_tokens
    parent = np.concatenate([D.chain(n) for n in n_new] + [[-1] * (T - sum(n_new))])
    parent = parent.astype(np.int64)
    d = rbkv.StepDraft(t).plan(i32(parent))
    tokens = rng.integers(0, 5, T)
    follow = np.concatenate([tokens[1:], [9]])           # (a chain's choices that all agree)
    half = np.where(rng.random(T) < 0.5, follow, 9)
    some = np.array([rng.integers(1, n + 1) if n else 0 for n in n_new])
    for chosen, given in ((tokens + 9, None), (follow, None), (half, None), (follow, some),
                          (tokens + 9, some), (half, None)):
        done = D.accept(want, parent, tokens, chosen, given, block)
        d.accept(i32(tokens), i32(chosen), None if given is None else i32(given))
        _kept(t, d, done)
    t.device_status()
    _built_again(rng, t, done, want, seen, n_new, block)


def test_two_drafts_of_one_step_accept(rbkv):
    """Another draft of the same step, planned and accepted after the first."""
    t, want, rng = _built(rbkv, [3, 40], [60, 50], block=8)
    parent = np.concatenate([D.chain(60), D.chain(50)])
    tokens = np.arange(t.max_tokens)
    for chosen in (tokens, tokens + 1, tokens):
        d = rbkv.StepDraft(t).plan(i32(parent))
        d.accept(i32(tokens), i32(chosen))
        done = D.accept(want, parent, tokens, chosen, None, 8)
        _kept(t, d, done)
    t.device_status()


# ---- released sequences ------------------------------------------------------------
@pytest.mark.parametrize("again", [False, True])
@pytest.mark.parametrize("seen,n_new", KEEP, ids=lambda x: str(len(x)))
def test_a_released_sequence_keeps_nothing(rbkv, seen, n_new, again):
    """Released between the build and the acceptance, or between two: its blocks stay free,
    its length 0, nothing of it is moved, and the next step may take its slot."""
    block, S = 8, len(n_new)
    t, want, rng = _built(rbkv, seen, n_new, block=block, seed=S, cfg=(8, 2, 64))
    T = t.max_tokens
    parent, tokens = random_trees(rng, n_new, T), np.zeros(T, np.int64)
    d = rbkv.StepDraft(t).plan(i32(parent))
    if again:
        d.accept(i32(tokens), i32(tokens))
    gone = np.arange(S) % 3 == 0
    t.release(i32(gone))
    done = D.accept(want, parent, tokens, tokens, None, block, released=np.flatnonzero(gone))
    caches = [torch.randn(t.config.cache_shape()) for _ in range(2)]
    dev = [c.cuda() for c in caches]
    d.accept(i32(tokens), i32(tokens))
    _kept(t, d, done)
    d.compact(*dev)
    for c, x in zip(caches, dev):
        D.compact(want, done, c, block)
        assert torch.equal(c, x.cpu())
    t.device_status()
    _built_again(rng, t, done, want, seen, n_new, block)


# ---- given tokens that are no chain --------------------------------------------------
@pytest.mark.parametrize("turned", [False, True])
@pytest.mark.parametrize("seen,n_new", KEEP + [([4, 9, 0], [3, 128, 33])],
                         ids=lambda x: str(len(x)))
def test_given_tokens_that_are_no_chain(rbkv, seen, n_new, turned):
    """Rows that were rotated by their places: a given token that does not follow the one
    before it would lie at another position than it was turned by.  So it, and what comes
    after it, is no longer given, and the status says so.  Rows as they came are kept as
    they are."""
    block = 8
    t, want, rng = _built(rbkv, seen, n_new, block=block, seed=7, cfg=(8, 2, 64))
    T, rows = t.max_tokens, int(want.q_start[-1])
    parent = random_trees(rng, n_new, T)
    tokens, chosen = rng.integers(0, 2, T), rng.integers(0, 2, T)
    caches = [torch.randn(t.config.cache_shape(), device="cuda") for _ in range(2)]
    q, k, v = (torch.randn(T, h, 64, device="cuda") for h in (8, 2, 2))
    d = rbkv.StepDraft(t)
    rope = rbkv.Rotary(64)
    for some in (np.array([min(n, 3) for n in n_new]), np.array([max(n - 1, min(n, 1)) for n in n_new]),
                 np.array(n_new)):
        d.plan(i32(parent))
        if turned:
            t.append_rotary(rope, q, k, v, *caches, draft=d)
        else:
            t.append(k, v, *caches)
        d.accept(i32(tokens), i32(chosen), i32(some))
        done = D.accept(want, parent, tokens, chosen, some, block, turned=turned)
        _kept(t, d, done)
        if not turned:
            t.device_status()
            continue
        place = d.place.cpu().numpy()
        for r in np.flatnonzero(done.path >= 0):
            assert place[done.path[r]] == want.position[r]
        if (D.accept(want, parent, tokens, chosen, some, block).path == done.path).all():
            t.device_status()
        else:
            assert _status(rbkv, t) == INVALID
    # a chain that is given is kept whole, with a chunk behind it
    chains = np.concatenate([D.chain(n) for n in n_new] + [[0] * (T - rows)]).astype(np.int64)
    d.plan(i32(chains))
    t.append_rotary(rope, q, k, v, *caches, draft=d)
    d.accept(i32(tokens), i32(tokens + 1), i32(n_new))
    t.device_status()
    assert d.accepted.tolist() == list(n_new)


def test_rows_turned_in_an_earlier_step(rbkv):
    """The rotation of the step before says nothing of this one's rows."""
    t, want, rng = _built(rbkv, [0], [4], block=8, pad=4, cfg=(8, 2, 64))
    caches = [torch.randn(t.config.cache_shape(), device="cuda") for _ in range(2)]
    q, k, v = (torch.randn(t.max_tokens, h, 64, device="cuda") for h in (8, 2, 2))
    d = rbkv.StepDraft(t)
    tree, tokens = i32([-1, 0, 0, 0] + [0] * (t.max_tokens - 4)), i32([0] * t.max_tokens)
    d.plan(tree)
    t.append_rotary(rbkv.Rotary(64), q, k, v, *caches, draft=d)
    d.accept(tokens, tokens + 1, i32([3]))
    assert d.accepted.tolist() == [2] and _status(rbkv, t) == INVALID
    t.build(t.ctx, i32([4]))
    d.plan(tree)
    t.append(k, v, *caches)
    d.accept(tokens, tokens + 1, i32([3]))
    t.device_status()
    assert d.accepted.tolist() == [3] and t.ctx.tolist() == [5]
