"""Drafted tokens of a step and rotary positions, in plain loops (oracle).

A sequence's new tokens form a tree (``parent[i] < i``, -1: none); a token sees
the cached ones and those on its way up.  After a choice at every token the path
that the choices agree with is kept.  A tree that is none is taken as a chain.
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import List

import numpy as np

from .step import Step

MAX_TREE = 128


def chain(n: int) -> List[int]:
    return list(range(-1, n - 1))


def parents_of(step: Step, parent, s: int):
    """(the tree of sequence s as it is taken, whether it was one)."""
    a, b = int(step.q_start[s]), int(step.q_start[s + 1])
    p = [int(x) for x in parent[a:b]]
    if all(-1 <= x < i for i, x in enumerate(p)) and (len(p) <= MAX_TREE or p == chain(len(p))):
        return p, True
    return chain(len(p)), False


def way_up(p, i: int) -> List[int]:
    """Token i and those that it follows, from the root."""
    out = []
    while i >= 0:
        out.append(i)
        i = p[i]
    return out[::-1]


@dataclass
class Plan:
    good: bool
    place: np.ndarray
    ancestors: np.ndarray      # [rows][4] uint32 as int32


def plan(step: Step, parent, max_tokens: int) -> Plan:
    place = np.full(max_tokens, -1)
    sets = np.zeros((max_tokens, 4), np.uint32)
    good = True
    for s in range(len(step.ctx)):
        p, ok = parents_of(step, parent, s)
        good &= ok
        q0, n = int(step.q_start[s]), len(p)
        seen = int(step.ctx[s]) - n
        for i in range(n):
            if n > MAX_TREE:
                place[q0 + i] = seen + i
                continue
            up = way_up(p, i)
            place[q0 + i] = seen + len(up) - 1
            for j in up:
                sets[q0 + i, j // 32] |= np.uint32(1) << np.uint32(j % 32)
    return Plan(good, place, sets.view(np.int32))


@dataclass
class Accepted:
    path: np.ndarray
    accepted: np.ndarray
    next_token: np.ndarray
    ctx: np.ndarray
    free: List[bool]


def accept(step: Step, parent, tokens, chosen, given, block_size: int, released=(),
           turned: bool = False) -> Accepted:
    """``released``: sequences given back since the build, which keep nothing.  ``turned``:
    the rows were rotated by their places, so that given tokens are kept as far as each
    follows the one before it."""
    S = len(step.ctx)
    path = np.full(len(tokens), -1)
    accepted, last = np.zeros(S, np.int64), np.full(S, -1)
    ctx, free = step.ctx.copy(), list(step.free)
    for s in range(S):
        p, _ = parents_of(step, parent, s)
        q0, n = int(step.q_start[s]), len(p)
        if n == 0:
            continue
        if s in released:
            ctx[s] = 0
            for c in range(-(-int(step.ctx[s]) // block_size)):
                free[int(step.table[s, c])] = True
            continue
        g = 1 if given is None else min(max(int(given[s]), 1), n)
        if turned:
            g = next((i for i in range(1, g) if p[i] != i - 1), g)
        kept = list(range(g))
        while True:
            at = kept[-1]
            found = [c for c in range(at + 1, n)
                     if p[c] == at and tokens[q0 + c] == chosen[q0 + at]]
            if not found:
                break
            kept.append(found[0])
        path[q0:q0 + len(kept)] = q0 + np.array(kept)
        accepted[s], last[s] = len(kept), chosen[q0 + kept[-1]]
        seen = int(step.ctx[s]) - n
        ctx[s] = seen + len(kept)
        for c in range(-(-int(ctx[s]) // block_size), -(-(seen + n) // block_size)):
            free[int(step.table[s, c])] = True
    return Accepted(path, accepted, last, ctx, free)


def compact(step: Step, done: Accepted, cache, block_size: int) -> None:
    """Moves the kept rows of a cache [blocks][heads][block][dim] in place."""
    old = cache.clone()
    for r, src in enumerate(done.path):
        if src >= 0:
            (b, i), (c, j) = divmod(int(step.slot[r]), block_size), \
                divmod(int(step.slot[src]), block_size)
            cache[b, :, i] = old[c, :, j]


def rotate(x, position, theta, layout: str, scale: float = 1.0) -> np.ndarray:
    """x [rows][heads][D] by the rows' positions: in long double (at least 64 bits of
    significand), so that far positions keep their angles; returned in fp64."""
    wide = np.longdouble
    R = 2 * len(theta)
    angle = np.asarray(position).astype(wide)[:, None] * np.asarray(theta).astype(wide)
    c, s = np.cos(angle)[:, None] * wide(scale), np.sin(angle)[:, None] * wide(scale)
    out = np.asarray(x, np.float64).astype(wide)
    a, b = (slice(0, R // 2), slice(R // 2, R)) if layout == "half" else \
        (slice(0, R, 2), slice(1, R, 2))
    u, v = out[..., a].copy(), out[..., b].copy()
    out[..., a], out[..., b] = u * c - v * s, v * c + u * s
    return out.astype(np.float64)
