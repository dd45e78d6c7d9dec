"""The operators of a serving step whose metadata lives on the GPU, as measured cases.

A step of a batch that shares one long prefix: block tables and slot maps are
built on the GPU from the requests' lengths, the new K/V rows are appended
through the slot map, and every row attends the shared prefix and its own
sequence's keys.  Token positions and block tables are those of a sequence's
own tokens; the prefix has a block list of its own.

``run`` computes each operator in its plain form, or calls the library when
``own`` is set.  Caches are [blocks][kv heads][block][dim], Q and O
[rows][heads][dim], query head h reads KV head h // (heads / kv heads).
"""
import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def _tables_case(name, decodes, own_hi, block, num_blocks, prompts=0, rows=0, idle=0, pad=0):
    return {"name": name, "op": "tables", "decodes": decodes, "own_lo": 1, "own_hi": own_hi,
            "prompts": prompts, "rows": rows, "cached": 0, "idle": idle, "pad": pad,
            "block": block, "num_blocks": num_blocks}


def _append_case(name, decodes, own_hi, block, hkv, dim, dtype, prompts=0, rows=0):
    return {"name": name, "op": "append", "decodes": decodes, "own_lo": 1, "own_hi": own_hi,
            "prompts": prompts, "rows": rows, "cached": 0, "idle": 0, "pad": 0, "block": block,
            "hq": hkv, "hkv": hkv, "dim": dim, "dtype": dtype}


def _attention_case(name, hq, hkv, dim, block, dtype, prefix, decodes, own_lo, own_hi, prompts=0,
                    rows=0, cached=0, idle=0, pad=0):
    return {"name": name, "op": "attention", "hq": hq, "hkv": hkv, "dim": dim, "block": block,
            "dtype": dtype, "prefix": prefix, "decodes": decodes, "own_lo": own_lo,
            "own_hi": own_hi, "prompts": prompts, "rows": rows, "cached": cached, "idle": idle,
            "pad": pad}


def listed():
    return [
        # a small decoding batch: the call's latency
        _tables_case("tables-16", 16, 256, 64, 1024),
        # 512 decoding requests of up to 8192 tokens
        _tables_case("tables-512", 512, 8192, 64, 49152),
        # the same with two prompt chunks, some idle request slots and spare rows
        _tables_case("tables-512-prompts", 512, 8192, 64, 49152, 2, 768, 30, 70),
        # thousands of requests in 16-token blocks: a million-block pool
        _tables_case("tables-4096", 4096, 8192, 16, 1300000, 8, 500),
        # K and V of one decoding step, and of a pass with prompt chunks
        _append_case("append-64", 64, 4096, 64, 8, 128, "bf16"),
        _append_case("append-2048", 512, 512, 64, 8, 128, "bf16", 2, 768),
        # a few short generations behind a system prompt, one query head per KV head
        _attention_case("attention-16", 32, 32, 128, 64, "bf16", 512, 16, 1, 120),
        # one request over a long document
        _attention_case("attention-1", 32, 8, 128, 64, "bf16", 32768, 1, 700, 700),
        # a full decoding batch behind a long prompt, groups of 4
        _attention_case("attention-512", 32, 8, 128, 64, "bf16", 4096, 512, 1, 512),
        # groups of 8, an odd prefix of the longest benchmark context
        _attention_case("attention-64", 64, 8, 128, 64, "bf16", 15999, 64, 128, 1024),
        # decoding requests with new user turns beside them, idle slots, spare rows
        _attention_case("attention-mixed", 32, 8, 128, 64, "bf16", 2300, 128, 1, 512, 8, 160, 33,
                        5, 60),
        # fp32, head dim 64, 16-token blocks
        _attention_case("attention-f32", 8, 2, 64, 16, "f32", 333, 32, 1, 100, 2, 21, 5),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["tables", "append", "attention", "attention", "attention"])
    block = rng.choice([16, 32, 64, 64, 128])
    if op == "tables":
        decodes, hi = _log_int(rng, 1, 4096), _log_int(rng, 16, 8192)
        prompts = rng.choice([0, 0, 1, 5])
        c = _tables_case("", decodes, hi, block, 0, prompts, _log_int(rng, 1, 500),
                         rng.randint(0, 9), rng.randint(0, 99))
        need = (decodes * (-(-hi // block)) + prompts * (-(-c["rows"] // block)))
        c["num_blocks"] = need + rng.randint(1, need + 1)
        while c["num_blocks"] > 1300000:   # the largest listed pool
            c["num_blocks"] = need + 1
            c["decodes"] = c["decodes"] * 3 // 4
            need = c["num_blocks"] = (c["decodes"] * (-(-hi // block)) +
                                      prompts * (-(-c["rows"] // block)) + 1)
    elif op == "append":
        c = _append_case("", _log_int(rng, 1, 512), _log_int(rng, 1, 512), block,
                         rng.choice([1, 2, 8]), rng.choice([64, 128]),
                         rng.choice(["bf16", "bf16", "f32"]), rng.choice([0, 1, 2]),
                         _log_int(rng, 1, 600))
    else:
        hq, hkv = rng.choice([(32, 32), (32, 8), (32, 8), (64, 8), (16, 1), (20, 4), (8, 2)])
        dim, dtype = rng.choice([(128, "bf16")] * 6 + [(64, "bf16"), (64, "f32")])
        c = _attention_case("", hq, hkv, dim, block, dtype,
                            rng.choice([0, 1, 2]) and _log_int(rng, 1, 16000),
                            _log_int(rng, 1, 512), 1, _log_int(rng, 1, 1024),
                            rng.choice([0, 0, 1, 4]), _log_int(rng, 2, 300),
                            rng.randint(0, 100), rng.randint(0, 5), rng.randint(0, 40))
        # no more work than the largest listed case; the CUDA-core shapes far less
        top = 3.0e10 if (dim, dtype) == (128, "bf16") else 1.0e9
        while work(c)["flops"] > top:
            c["decodes"] = max(1, c["decodes"] // 2)
            c["prompts"] = min(c["prompts"], 1)
            c["prefix"] = c["prefix"] * 3 // 4
    del c["name"]
    return c


def _lengths(c, rng):
    """(seen, n_new) of the batch's request slots, in a seeded order.  Prompt
    chunks of an attention step are ragged; the other cases fill every row."""
    n, p, idle = c["decodes"], c["prompts"], c["idle"]
    seen = np.concatenate([rng.integers(c["own_lo"], c["own_hi"] + 1, n) - 1,
                           np.full(p, c["cached"]), rng.integers(0, c["own_hi"] + 1, idle)])
    rows = np.full(p, c["rows"])
    if c["op"] == "attention":
        rows = rng.integers((c["rows"] + 1) // 2, c["rows"] + 1, p)
    n_new = np.concatenate([np.ones(n, np.int64), rows, np.zeros(idle, np.int64)])
    order = rng.permutation(n + p + idle)
    return seen[order].astype(np.int64), n_new[order].astype(np.int64)


def _max_blocks(c):
    longest = max(c["own_hi"], c["cached"] + c["rows"] if c["prompts"] else 0)
    return -(-longest // c["block"]) + 1


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(a.astype(np.int32))).cuda()


def prepare(case, seed):
    c = case
    rng = np.random.default_rng([seed, 7])
    B = c["block"]
    seen, n_new = _lengths(c, rng)
    S, MB = len(seen), _max_blocks(c)
    held = -(-seen // B)
    after = int((-(-(seen + n_new) // B)).sum())
    pre_blocks = -(-c["prefix"] // B) if c["op"] == "attention" else 0
    num_blocks = after + pre_blocks + 16
    if c["op"] == "tables":
        num_blocks = c["num_blocks"]
    elif c["op"] == "append":   # the caches are outputs: their size goes by the case
        num_blocks = S * MB
    perm = rng.permutation(num_blocks)
    prefix_ids, perm = perm[:pre_blocks], perm[pre_blocks:]
    col = np.arange(MB)
    at = (np.cumsum(held) - held)[:, None] + col
    table = np.where(col < held[:, None], perm[np.minimum(at, len(perm) - 1)], -1)
    bits = np.zeros(-(-num_blocks // 32) * 32, np.uint8)
    bits[:num_blocks] = 1
    bits[prefix_ids] = 0
    bits[perm[:int(held.sum())]] = 0
    free = np.packbits(bits, bitorder="little").view("<u4").astype(np.int64)
    capacity = c["decodes"] + c["prompts"] * c["rows"] + c["pad"]
    s = {"case": c, "num_blocks": num_blocks, "capacity": capacity,
         "seen": _int32(seen), "n_new": _int32(n_new), "table": _int32(table),
         "free": _int32(np.where(free >= 2 ** 31, free - 2 ** 32, free))}
    if own:
        import ragged_blocked_kv_gb300 as rbkv
        cfg = rbkv.Config(c.get("hq", 1), c.get("hkv", 1), c.get("dim", 128), B,
                          c.get("dtype", "bf16"), num_blocks)
        s["tables"] = rbkv.StepTables(cfg, S, MB, capacity)
    if c["op"] == "tables":
        return s
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    cache = (num_blocks, c["hkv"], B, c["dim"])
    s["k_cache"], s["v_cache"] = normal(*cache), normal(*cache)
    if own:
        s["tables"].build(s["seen"], s["n_new"], block_table=s["table"], free=s["free"])
    s["built"] = _tables_plain(s)
    if c["op"] == "append":
        s["k_new"] = normal(capacity, c["hkv"], c["dim"])
        s["v_new"] = normal(capacity, c["hkv"], c["dim"])
        return s
    s["q"] = normal(capacity, c["hq"], c["dim"])
    s["o"] = torch.zeros_like(s["q"])
    s["prefix"] = _int32(prefix_ids)
    s["longest"] = int((seen + n_new)[n_new > 0].max())
    if own:
        s["workspace"] = torch.empty(max(256, s["tables"].workspace_bytes(c["prefix"])),
                                     dtype=torch.uint8, device="cuda")
    return s


def _tables_plain(s):
    """Blocks in sequence order, lowest free id first; nothing is scheduled
    where the step does not fit its rows, its table or the pool."""
    B, nb, T = s["case"]["block"], s["num_blocks"], s["capacity"]
    seen, n_new, table = s["seen"].long(), s["n_new"].long(), s["table"]
    dev = seen.device
    shift = torch.arange(32, device=dev)
    bits = ((s["free"].long()[:, None] >> shift) & 1).reshape(-1)
    held = (seen + B - 1) // B
    need = (seen + n_new + B - 1) // B
    ok = ((n_new.sum() <= T) & (need <= table.shape[1]).all() &
          ((need - held).sum() <= bits.sum()))
    n_new = torch.where(ok, n_new, 0)
    need = torch.where(ok, need, held)
    ctx = seen + n_new
    q_start = torch.nn.functional.pad(torch.cumsum(n_new, 0), (1, 0))
    rank = torch.cumsum(bits, 0) - 1
    every = torch.arange(bits.numel(), device=dev)
    ids = torch.zeros(bits.numel() + 1, dtype=torch.long, device=dev)
    ids.scatter_(0, torch.where(bits == 1, rank, bits.numel()), every)
    grow = need - held
    first = torch.cumsum(grow, 0) - grow
    col = torch.arange(table.shape[1], device=dev)
    k = first[:, None] + col - held[:, None]
    taken = (col >= held[:, None]) & (col < need[:, None])
    table = torch.where(taken, ids[k.clamp(0, bits.numel())], table.long())
    bits = bits * (rank >= grow.sum())
    word = (bits.reshape(-1, 32) << shift).sum(1)
    free = torch.where(word >= 2 ** 31, word - 2 ** 32, word)
    row = torch.arange(T, device=dev)
    live = row < q_start[-1]
    seq = torch.searchsorted(q_start[1:].contiguous(), row, right=True).clamp(max=len(seen) - 1)
    pos = seen[seq] + row - q_start[seq]
    blk = table[seq, (pos // B).clamp(0, table.shape[1] - 1)]
    out = {"block_table": table, "free": free, "ctx": ctx, "q_start": q_start,
           "position": torch.where(live, pos, -1),
           "slot": torch.where(live, blk * B + pos % B, -1)}
    out = {k: v.to(torch.int32) for k, v in out.items()}
    s["seq"] = seq
    return out


def _append_plain(s):
    B, slot = s["case"]["block"], s["built"]["slot"].long()
    s["k_cache"][slot // B, :, slot % B] = s["k_new"]
    s["v_cache"][slot // B, :, slot % B] = s["v_new"]
    return [s["k_cache"], s["v_cache"]]


def _gather(cache, table, length):
    """Rows 0 .. length-1 of the sequences of a block table: [S, length, kv heads, dim]."""
    B = cache.shape[2]
    pos = torch.arange(length, device=cache.device)
    blk = table.long()[:, pos // B].clamp(min=0)
    return cache[blk, :, pos % B].float()


def _attention_plain(s):
    c, t = s["case"], s["built"]
    T, hkv, dim = s["capacity"], c["hkv"], c["dim"]
    g = c["hq"] // hkv
    q = s["q"].float().reshape(T, hkv, g, dim) * dim ** -0.5
    k_own = _gather(s["k_cache"], t["block_table"], s["longest"])[s["seq"]]
    score = torch.matmul(q, k_own.permute(0, 2, 3, 1))
    visible = torch.arange(s["longest"], device=q.device) <= t["position"][:, None]
    score = torch.where(visible[:, None, None], score, float("-inf"))
    P = c["prefix"]
    k_pre = _gather(s["k_cache"], s["prefix"][None], P)[0]
    v_pre = _gather(s["v_cache"], s["prefix"][None], P)[0]
    rows = q.permute(1, 0, 2, 3).reshape(hkv, T * g, dim)
    pre = torch.matmul(rows, k_pre.permute(1, 2, 0)).reshape(hkv, T, g, P).permute(1, 0, 2, 3)
    score = torch.cat([pre, score], -1)
    top = score.amax(-1, keepdim=True)
    score = torch.exp(score - torch.where(top == float("-inf"), 0, top))
    total = score.sum(-1, keepdim=True)
    v_own = _gather(s["v_cache"], t["block_table"], s["longest"])[s["seq"]]
    out = torch.matmul(score[..., P:], v_own.permute(0, 2, 1, 3))
    rows = score[..., :P].permute(1, 0, 2, 3).reshape(hkv, T * g, P)
    out = out + torch.matmul(rows, v_pre.permute(1, 0, 2)).reshape(hkv, T, g, dim).transpose(0, 1)
    out = (out / total).reshape(T, c["hq"], dim).to(s["o"].dtype)
    live = (t["position"] >= 0)[:, None, None]
    return torch.where(live, out, s["o"])


def run(state):
    s, op = state, state["case"]["op"]
    if op == "tables":
        if own:
            t = s["tables"].build(s["seen"], s["n_new"], block_table=s["table"], free=s["free"])
            return {"block_table": t.block_table, "free": t.free, "ctx": t.ctx,
                    "q_start": t.q_start, "position": t.position, "slot": t.slot}
        return _tables_plain(s)
    if op == "append":
        if own:
            s["tables"].append(s["k_new"], s["v_new"], s["k_cache"], s["v_cache"])
            return [s["k_cache"], s["v_cache"]]
        return _append_plain(s)
    if own:
        return s["tables"].attention(s["q"], s["k_cache"], s["v_cache"], prefix_table=s["prefix"],
                                     prefix_len=s["case"]["prefix"], o=s["o"],
                                     workspace=s["workspace"])
    return _attention_plain(s)


def work(case):
    """One pass at the mean lengths of the case's distribution."""
    c = case
    S = c["decodes"] + c["prompts"] + c["idle"]
    rows_each = 0.75 * c["rows"] if c["op"] == "attention" else c["rows"]
    T = c["decodes"] + c["prompts"] * rows_each
    if c["op"] == "tables":
        table = S * _max_blocks(c) * 4
        bits = c["num_blocks"] / 8
        return {"bytes": int(2 * table + 2 * bits + 16 * S + 8 * (T + c["pad"])),
                "flops": int(S * _max_blocks(c) + c["num_blocks"] + T)}
    size = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "append":
        return {"bytes": int(4 * T * c["hkv"] * c["dim"] * size + 4 * T), "flops": int(T)}
    mean = (c["own_lo"] + c["own_hi"]) / 2
    own_keys = c["decodes"] * mean + c["prompts"] * (c["cached"] + rows_each)
    pairs = (c["decodes"] * (c["prefix"] + mean) +
             c["prompts"] * rows_each * (c["prefix"] + c["cached"] + rows_each / 2))
    return {"bytes": int((2 * (c["prefix"] + own_keys) * c["hkv"] + 2 * T * c["hq"]) *
                         c["dim"] * size),
            "flops": int(4 * c["dim"] * c["hq"] * pairs)}


def exact(case, seed):
    """Attention by sequence in 64 bits; tables and appends are whole numbers and copies."""
    if case["op"] != "attention":
        return None
    s = prepare(case, seed)
    B, g, dim = case["block"], case["hq"] // case["hkv"], case["dim"]
    table = s["built"]["block_table"].cpu().numpy()
    seen, n_new = s["seen"].cpu().numpy(), s["n_new"].cpu().numpy()
    prefix = s["prefix"].cpu().numpy()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")

    def keys(cache, ids, n):
        picked = cache[torch.from_numpy(ids.astype(np.int64)).cuda()].double()
        return picked.transpose(1, 2).reshape(-1, case["hkv"], dim)[:n].transpose(0, 1)

    k_pre, v_pre = (keys(x, prefix, case["prefix"]) for x in (s["k_cache"], s["v_cache"]))
    row = 0
    for i in range(len(seen)):
        n, ctx = int(n_new[i]), int(seen[i] + n_new[i])
        if n == 0:
            continue
        ids = table[i, :-(-ctx // B)]
        k = torch.cat([k_pre, keys(s["k_cache"], ids, ctx)], 1)
        v = torch.cat([v_pre, keys(s["v_cache"], ids, ctx)], 1)
        q = s["q"][row:row + n].double().view(n, case["hkv"], g, dim).permute(1, 2, 0, 3)
        logit = q @ k[:, None].transpose(-1, -2) / dim ** 0.5
        last = case["prefix"] + int(seen[i]) + torch.arange(n, device="cuda")[:, None]
        hidden = torch.arange(k.shape[1], device="cuda")[None] > last
        prob = torch.softmax(logit.masked_fill(hidden, float("-inf")), -1)
        out[row:row + n] = (prob @ v[:, None]).permute(2, 0, 1, 3).reshape(n, case["hq"], dim)
        row += n
    return out
