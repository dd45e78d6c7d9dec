"""Seeded trees, a vectorised fp64 reference and error bounds for the tests of
drafted tokens and rotary positions (test infrastructure)."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle


def random_tree(rng, n):
    """Parents of n tokens: a chain, a bush, a random tree or a forest."""
    kind = rng.integers(0, 4)
    if kind == 0:
        return oracle.draft.chain(n)
    if kind == 1:
        return [-1 if i == 0 else (i - 1) // 3 for i in range(n)]
    low = -1 if kind == 3 else 0
    return [-1 if i == 0 else int(rng.integers(low, i)) for i in range(n)]


def random_trees(rng, n_new, rows):
    """parent [rows] (chains where there are more tokens than a tree may have)."""
    out = [p for n in n_new for p in (random_tree(rng, int(n)) if n <= oracle.draft.MAX_TREE
                                      else oracle.draft.chain(int(n)))]
    return np.array(out + [rng.integers(-9, 9) for _ in range(rows - len(out))], np.int64)


def draft_reference(step, parent, q, k_cache, v_cache, prefix_table, prefix_len):
    """As step_harness.reference, for a step of drafted tokens: fp64 O, sum_i w_i |v_i|,
    max_i sum_d |q_d k_id| / sqrt(D) over what a row sees, and the number of those keys."""
    T, (H_q, D) = int(step.q_start[-1]), q.shape[1:]
    H_kv, B = k_cache.shape[1:3]
    g = H_q // H_kv
    out = torch.zeros(T, H_q, D, dtype=torch.float64)
    absv, absqk = torch.zeros_like(out), torch.zeros(T, H_q, 1, dtype=torch.float64)
    keys = torch.zeros(T, 1, 1, dtype=torch.float64)

    def rows(cache, ids, n):
        ids = torch.as_tensor(np.asarray(ids).astype(np.int64))
        return cache[ids].double().transpose(1, 2).reshape(-1, H_kv, D)[:n]

    kp, vp = (rows(c, np.asarray(prefix_table)[:-(-prefix_len // B)], prefix_len)
              for c in (k_cache, v_cache))
    for s in range(len(step.ctx)):
        a, b = int(step.q_start[s]), int(step.q_start[s + 1])
        if a == b:
            continue
        n, first = int(step.ctx[s]), prefix_len + int(step.ctx[s]) - (b - a)
        ids = step.table[s][:-(-n // B)]
        k = torch.cat([kp, rows(k_cache, ids, n)]).permute(1, 2, 0)
        v = torch.cat([vp, rows(v_cache, ids, n)]).transpose(0, 1)
        p, _ = oracle.draft.parents_of(step, parent, s)
        sees = torch.zeros(b - a, prefix_len + n, dtype=torch.bool)
        sees[:, :first] = True
        for i in range(b - a):
            sees[i, [first + j for j in oracle.draft.way_up(p, i)]] = True
        used = sees.any(0)        # (a key that no row sees may hold anything)
        k = torch.where(used, k, 0.0)
        v = torch.where(used[:, None], v, 0.0)
        qs = q[a:b].double().reshape(b - a, H_kv, g, D).permute(1, 2, 0, 3)
        x = qs @ k[:, None] / math.sqrt(D)
        w = torch.softmax(x.masked_fill(~sees, -math.inf), -1)

        def back(y):
            return y.permute(2, 0, 1, 3).reshape(b - a, H_q, -1)

        out[a:b] = back(w @ v[:, None])
        absv[a:b] = back(w @ v.abs()[:, None])
        ax = (qs.abs() @ k.abs()[:, None] / math.sqrt(D)).masked_fill(~sees, 0.0)
        absqk[a:b] = back(ax.amax(-1, keepdim=True))
        keys[a:b, 0, 0] = sees.sum(1).double()
    return out, absv, absqk, keys


def rotary_bound(x, position, theta, layout, scale, exact, dtype):
    """Largest |computed - exact| of a rotation, per element.

    With u = 2^-24: the angle's fraction of a half turn is rounded to fp32 (at most
    u / 2 half turns, pi u / 2 of angle) and its table entry to fp64, twice (2^-52 of
    the angle itself); the sine and the cosine are off by two units in the last place
    (2 * 2^-23 at most); the product with the scale and the two products and the sum
    of a rotation are four more roundings.  All of that is relative to |x| + |y| of the
    pair, times the scale:
        (pi / 2 + 4 + 4) u + 2^-51 |angle| <= 10 u + 2^-51 |angle|.
    Then the output's own rounding: 2^-8 of it (bf16) or 2^-24 (fp32)."""
    u = 2.0 ** -24
    R = 2 * len(theta)
    x = np.asarray(x, np.float64)
    bound = np.zeros_like(x)
    angle = np.abs(np.asarray(position, np.float64)[:, None] * np.asarray(theta))[:, None]
    a, b = (slice(0, R // 2), slice(R // 2, R)) if layout == "half" else \
        (slice(0, R, 2), slice(1, R, 2))
    pair = (np.abs(x[..., a]) + np.abs(x[..., b])) * abs(scale) * (10 * u + 2.0 ** -51 * angle)
    bound[..., a] = bound[..., b] = pair
    out = 2.0 ** -8 if dtype == "bf16" else u
    return bound * (1 + 2 * out) + out * np.abs(exact) * (np.arange(x.shape[-1]) < R) + 1e-37
