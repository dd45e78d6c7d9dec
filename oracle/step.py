"""A step built from lengths, and attention with a shared prefix, in plain
loops and fp64 (oracle).

Block ids follow the composer's rule (lowest free id first, in sequence
order); a step that does not fit schedules nothing.  Attention is the
definition: one softmax over the prefix's keys and the sequence's own keys up
to the row's position (FastGen guide, Step 3's unsplit path).
"""
from __future__ import annotations

import math
from dataclasses import dataclass
from typing import List

import numpy as np


@dataclass
class Step:
    status: int                # 0, or the library's status of a step that does not fit
    q_start: np.ndarray
    ctx: np.ndarray
    table: np.ndarray
    free: List[bool]
    position: np.ndarray
    slot: np.ndarray


def build(seen, n_new, table, free, block_size: int, max_tokens: int) -> Step:
    """``free``: one truth value per block.  ``table``: [S][max_blocks]."""
    seen, n_new = [int(x) for x in seen], [int(x) for x in n_new]
    S, max_blocks = table.shape
    table, free = table.copy(), list(free)
    empty = Step(0, np.zeros(S + 1, np.int64), np.array(seen), table.copy(), list(free),
                 np.full(max_tokens, -1), np.full(max_tokens, -1))
    need = [-(-(a + b) // block_size) for a, b in zip(seen, n_new)]
    if min(seen) < 0 or min(n_new) < 0:
        empty.status = -1
        return empty
    if sum(n_new) > max_tokens or max(need) > max_blocks:
        empty.status = -6
        return empty
    if sum(n - -(-a // block_size) for n, a in zip(need, seen)) > sum(free):
        empty.status = -2
        return empty
    out = empty
    row = 0
    for s in range(S):
        for c in range(-(-seen[s] // block_size), need[s]):
            b = free.index(True)
            free[b] = False
            table[s, c] = b
        for j in range(n_new[s]):
            p = seen[s] + j
            out.position[row] = p
            out.slot[row] = table[s, p // block_size] * block_size + p % block_size
            row += 1
        out.q_start[s + 1] = row
    out.ctx = np.array(seen) + np.array(n_new)
    out.table, out.free = table, free
    return out


def attention(step: Step, q, k_cache, v_cache, prefix_table, prefix_len: int) -> np.ndarray:
    """q [rows][H_q][D], caches [blocks][H_kv][B][D], all fp64; rows of the step."""
    H_q, D = q.shape[1:]
    H_kv, B = k_cache.shape[1:3]
    g = H_q // H_kv
    T = int(step.q_start[-1])
    out = np.zeros((T, H_q, D))

    def rows(cache, ids, n):
        return np.stack([cache[ids[i // B], :, i % B] for i in range(n)]) if n else \
            np.zeros((0, H_kv, D))

    kp, vp = (rows(c, prefix_table, prefix_len) for c in (k_cache, v_cache))
    for s in range(len(step.ctx)):
        a, b = int(step.q_start[s]), int(step.q_start[s + 1])
        if a == b:
            continue
        n = int(step.ctx[s])
        k = np.concatenate([kp, rows(k_cache, step.table[s], n)])
        v = np.concatenate([vp, rows(v_cache, step.table[s], n)])
        for r in range(a, b):
            m = prefix_len + int(step.position[r]) + 1
            for h in range(H_q):
                x = k[:m, h // g] @ q[r, h] / math.sqrt(D)
                w = np.exp(x - x.max())
                out[r, h] = w @ v[:m, h // g] / w.sum()
    return out
