"""Seeded steps, a vectorised fp64 reference and derived error bounds for the
tests of device-built steps (test infrastructure)."""
from __future__ import annotations

import math

import numpy as np
import torch

import oracle


def free_words(free) -> np.ndarray:
    """One truth value per block -> int32 words, bit i of word w = block 32 w + i."""
    bits = np.zeros(-(-len(free) // 32) * 32, np.uint8)
    bits[:len(free)] = free
    return np.packbits(bits, bitorder="little").view("<u4").astype(np.uint32).view(np.int32)


def random_batch(rng, seen, block_size, max_blocks, num_blocks, reserved=0):
    """A table holding ceil(seen / B) random distinct blocks per sequence, the
    free map, and `reserved` further blocks that are neither free nor held."""
    seen = np.asarray(seen)
    held = -(-seen // block_size)
    perm = rng.permutation(num_blocks)
    assert held.sum() + reserved <= num_blocks
    table = np.full((len(seen), max_blocks), -1, np.int64)
    at = reserved
    for s, n in enumerate(held):
        table[s, :n] = perm[at:at + n]
        at += n
    free = np.zeros(num_blocks, bool)
    free[perm[at:]] = True
    return table, free, perm[:reserved]


def i32(a, device="cuda"):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).to(device)


def reference(step: oracle.step.Step, q, k_cache, v_cache, prefix_table, prefix_len):
    """fp64 (torch, CPU): O, sum_i w_i |v_i| and max_i sum_d |q_d k_id| / sqrt(D)
    per row, head (and dim), of the step's rows."""
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
        n = int(step.ctx[s])
        ids = step.table[s][:-(-n // B)]
        k = torch.cat([kp, rows(k_cache, ids, n)]).permute(1, 2, 0)      # [H_kv, D, keys]
        v = torch.cat([vp, rows(v_cache, ids, n)]).transpose(0, 1)       # [H_kv, keys, D]
        qs = q[a:b].double().reshape(b - a, H_kv, g, D).permute(1, 2, 0, 3)
        x = qs @ k[:, None] / math.sqrt(D)
        last = prefix_len + torch.as_tensor(step.position[a:b].astype(np.int64))
        hidden = torch.arange(k.shape[2])[None] > last[:, None]
        w = torch.softmax(x.masked_fill(hidden, -math.inf), -1)

        def back(y):
            return y.permute(2, 0, 1, 3).reshape(b - a, H_q, -1)

        out[a:b] = back(w @ v[:, None])
        absv[a:b] = back(w @ v.abs()[:, None])
        ax = (qs.abs() @ k.abs()[:, None] / math.sqrt(D)).masked_fill(hidden, 0.0)
        absqk[a:b] = back(ax.amax(-1, keepdim=True))
        keys[a:b, 0, 0] = last.double() + 1
    return out, absv, absqk, keys


def error_bound(ref, D: int, dtype: str):
    """Largest |computed - exact| per element.

    With u = 2^-24 (fp32): a score, scaled into base 2 (its scale is one more
    rounding), is off by at most (D + 4) u sum|q k| / sqrt(D); exponentials of
    that, 2^-22 each for the exponential itself and as much for the running
    maximum's corrections, and sums of n terms in some order make every weight
    off by a factor within 1 +- d, numerator and denominator alike:
        d = 2 ((D + 4) u max|q||k| + 2^-20 + (n + 64) u).
    bf16: the weights are rounded before the value product (2^-8 each), the
    output once (2^-8 of itself); fp32: the output once (2^-24).
    """
    out, absv, absqk, keys = ref
    u = 2.0 ** -24
    d = 2 * ((D + 4) * u * absqk + 2.0 ** -20 + (keys + 64) * u)
    if dtype == "bf16":
        return (2.0 ** -8 + d) * absv * (1 + 2.0 ** -8) + 2.0 ** -8 * out.abs()
    return d * absv * (1 + 2.0 ** -20) + u * out.abs()
