"""The operators of a step with rotated keys and drafted tokens, as measured cases.

A step whose sequences each take a tree of drafted tokens (several candidate
continuations at once): Q and K are rotated by the tokens' positions as K and V
are appended, the trees' ancestor sets are worked out once, every token attends
the shared prefix, its sequence's cached keys and its own ancestors, and then the
drawn path is kept: lengths are cut back, blocks returned, and the kept rows of
K and V moved together.

``run`` computes each operator in its plain form, or calls the library when
``own`` is set.  Caches are [blocks][kv heads][block][dim], Q and O
[rows][heads][dim], query head h reads KV head h // (heads / kv heads).
"""
import math

import numpy as np
import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
_MAX_NODES = 128            # tokens of a tree; longer runs of new tokens are chains


def _rotary_case(name, decodes, own_hi, block, hq, hkv, dim, rot, layout, dtype, prompts=0, rows=0,
                 prefix=0, base=10000.0, factor=1.0, scaling="none", pad=0):
    return {"name": name, "op": "rotary", "decodes": decodes, "own_hi": own_hi, "nodes": 1,
            "prompts": prompts, "rows": rows, "idle": 0, "pad": pad, "block": block, "hq": hq,
            "hkv": hkv, "dim": dim, "rot": rot, "layout": layout, "dtype": dtype,
            "prefix": prefix, "base": base, "factor": factor, "scaling": scaling}


def _draft_case(name, decodes, nodes, prompts=0, rows=0, idle=0, pad=0):
    return {"name": name, "op": "draft", "decodes": decodes, "own_hi": 300, "nodes": nodes,
            "prompts": prompts, "rows": rows, "idle": idle, "pad": pad, "block": 64, "hq": 1,
            "hkv": 1, "dim": 128, "dtype": "bf16", "prefix": 0}


def _tree_case(name, decodes, nodes, own_lo, own_hi, block, hq, hkv, dim, dtype, prefix=0,
               prompts=0, rows=0, idle=0, pad=0):
    return {"name": name, "op": "tree", "decodes": decodes, "own_lo": own_lo, "own_hi": own_hi,
            "nodes": nodes, "prompts": prompts, "rows": rows, "idle": idle, "pad": pad,
            "block": block, "hq": hq, "hkv": hkv, "dim": dim, "dtype": dtype, "prefix": prefix}


def _accept_case(name, decodes, nodes, own_hi, block, hkv, dim, dtype, prompts=0, rows=0, idle=0):
    return {"name": name, "op": "accept", "decodes": decodes, "own_hi": own_hi, "nodes": nodes,
            "prompts": prompts, "rows": rows, "idle": idle, "pad": 0, "block": block, "hq": hkv,
            "hkv": hkv, "dim": dim, "dtype": dtype, "prefix": 0}


def listed():
    return [
        # one token of a small decoding batch: the call's latency
        _rotary_case("rotary-16", 16, 4096, 64, 32, 8, 128, 128, "half", "bf16"),
        # a full pass: a decoding batch and two prompt chunks behind a system prompt, a context
        # stretched to eight times its length
        _rotary_case("rotary-2048", 512, 512, 64, 32, 8, 128, 128, "half", "bf16", 2, 768, 2300,
                     500000.0, 8.0, "parts"),
        # fp32, a quarter of the head rotated, neighbouring pairs, spare rows
        _rotary_case("rotary-partial", 100, 300, 16, 8, 8, 64, 16, "interleaved", "f32", 1, 301,
                     pad=20),
        # a small batch's trees: the call's latency
        _draft_case("draft-16", 16, 8),
        # large trees of a large batch, beside prompt chunks and idle slots
        _draft_case("draft-512", 512, 64, 2, 768, 9, 60),
        # a few short generations with trees of eight
        _tree_case("tree-8", 8, 8, 1, 512, 64, 32, 32, 128, "bf16"),
        # one request over a long document
        _tree_case("tree-1", 1, 64, 32768, 32768, 64, 32, 8, 128, "bf16"),
        # a batch of long contexts, groups of 4
        _tree_case("tree-64", 64, 32, 1, 8192, 64, 32, 8, 128, "bf16"),
        # short trees of a decoding batch behind a shared prompt, prompt chunks, idle slots
        _tree_case("tree-mixed", 96, 6, 1, 1024, 64, 64, 8, 128, "bf16", 2300, 2, 500, 5, 40),
        # fp32, head dim 64, 16-token blocks
        _tree_case("tree-f32", 8, 13, 1, 300, 16, 8, 2, 64, "f32", 77, 1, 21),
        # a small batch's verdicts
        _accept_case("accept-16", 16, 8, 1024, 64, 8, 128, "bf16"),
        # large trees of a large batch
        _accept_case("accept-256", 256, 60, 1024, 64, 8, 128, "bf16", 2, 100, 7),
    ]


def _log_int(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["rotary", "rotary", "draft", "tree", "tree", "tree", "accept"])
    block = rng.choice([16, 32, 64, 64, 128])
    prompts = rng.choice([0, 0, 1, 2])
    dim, dtype = rng.choice([(128, "bf16")] * 6 + [(64, "bf16"), (64, "f32")])
    if op == "rotary":
        rot = rng.choice([dim, dim, dim // 2, dim // 4, 20])
        scaling = rng.choice(["none", "linear", "base", "parts"])
        c = _rotary_case("", _log_int(rng, 1, 512), _log_int(rng, 1, 512), block,
                         *rng.choice([(32, 32), (32, 8), (64, 8), (8, 1)]), dim, rot,
                         rng.choice(["half", "half", "interleaved"]), dtype, min(prompts, 1),
                         _log_int(rng, 1, 768), rng.choice([0, _log_int(rng, 1, 100000)]),
                         rng.choice([10000.0, 500000.0]),
                         1.0 if scaling == "none" else rng.choice([2.0, 4.5, 8.0]), scaling,
                         rng.randint(0, 50))
    elif op == "draft":
        c = _draft_case("", _log_int(rng, 1, 512), _log_int(rng, 1, 64), prompts,
                        _log_int(rng, 1, 768), rng.randint(0, 9), rng.randint(0, 99))
    elif op == "accept":
        c = _accept_case("", _log_int(rng, 1, 256), _log_int(rng, 1, 100), _log_int(rng, 1, 1024),
                         block, rng.choice([1, 2, 8]), dim, dtype, prompts,
                         _log_int(rng, 1, 100), rng.randint(0, 7))
        while c["decodes"] * c["nodes"] > 256 * 60:
            c["nodes"] //= 2
    else:
        hq, hkv = rng.choice([(32, 32), (32, 8), (32, 8), (64, 8), (16, 1), (20, 4), (8, 2)])
        hi = _log_int(rng, 1, 8192)
        c = _tree_case("", _log_int(rng, 1, 128), _log_int(rng, 1, 100), rng.choice([1, hi]), hi,
                       block, hq, hkv, dim, dtype, rng.choice([0, 0, _log_int(rng, 1, 8000)]),
                       prompts, _log_int(rng, 1, 500), rng.randint(0, 5), rng.randint(0, 40))
        # no more work than the largest listed case; the CUDA-core shapes far less
        top = 3.0e10 if (dim, dtype) == (128, "bf16") else 2.0e8
        while work(c)["flops"] > top or work(c)["bytes"] > 1.0e9:
            c["decodes"] = max(1, c["decodes"] // 2)
            c["nodes"] = max(1, c["nodes"] * 3 // 4)
            c["own_lo"], c["own_hi"] = -(-c["own_lo"] * 3 // 4), -(-c["own_hi"] * 3 // 4)
            c["rows"] = max(1, c["rows"] * 3 // 4)
            c["prefix"] = c["prefix"] * 3 // 4
    del c["name"]
    return c


# ---- inputs ----------------------------------------------------------------------
def _lengths(c, rng):
    """(seen, n_new, drafted) of the request slots, in a seeded order: trees of
    between half of the nodes and all of them, prompt chunks, idle slots."""
    n, p, idle = c["decodes"], c["prompts"], c["idle"]
    seen = np.concatenate([rng.integers(c.get("own_lo", 1), c["own_hi"] + 1, n),
                           rng.integers(0, 40, p), rng.integers(0, c["own_hi"] + 1, idle)])
    trees = rng.integers((c["nodes"] + 1) // 2, c["nodes"] + 1, n)
    chunks = np.full(p, c["rows"])
    if c["op"] == "rotary":        # (every row of the step, but for the spare ones)
        trees = np.ones(n, np.int64)
    n_new = np.concatenate([trees, chunks, np.zeros(idle, np.int64)])
    drafted = np.concatenate([np.ones(n, bool), np.zeros(p + idle, bool)])
    order = rng.permutation(n + p + idle)
    return seen[order].astype(np.int64), n_new[order].astype(np.int64), drafted[order]


def _parents(n, branches):
    """A tree in level order with `branches` children per token (1: a chain)."""
    return np.maximum(-1, (np.arange(n) + branches - 1) // branches - 1)


def _path(parent, rng):
    """A path of the tree from its root.  Its tokens are in their places already, or
    past the path's end, so that moving them there a second time changes nothing."""
    n = len(parent)
    node, up = int(rng.integers(0, n)), []
    while node >= 0:
        up.append(node)
        node = int(parent[node])
    up = up[::-1]
    while any(p != d and p < len(up) for d, p in enumerate(up)):
        up.pop()
    return up


def _int32(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a).astype(np.int32))).cuda()


def _inv_freq(c):
    """Angle per position of every pair of elements, in 64 bits."""
    R, base, f = c["rot"], c["base"], c["factor"]
    if c["scaling"] == "base":
        base = base * f ** (R / max(R - 2, 1))
    theta = base ** (-np.arange(0, R, 2, dtype=np.float64) / R)
    if c["scaling"] == "linear":
        theta = theta / f
    if c["scaling"] == "parts":
        r = 8192 * theta / (2 * math.pi)
        keep = np.clip((r - 1.0) / (32.0 - 1.0), 0.0, 1.0)
        theta = theta * (keep + (1.0 - keep) / f)
    return theta


def prepare(case, seed):
    c = case
    rng = np.random.default_rng([seed, 11])
    B = c["block"]
    seen, n_new, drafted = _lengths(c, rng)
    S = len(seen)
    MB = max(1, -(-(c["own_hi"] + max(c["nodes"], 40 + c["rows"])) // B))
    held, need = -(-seen // B), -(-(seen + n_new) // B)
    pre_blocks = -(-c["prefix"] // B) if c["op"] == "tree" else 0
    num_blocks = S * MB + pre_blocks       # (the caches are outputs: their size goes by the case)
    if c["op"] == "tree":
        num_blocks = int(need.sum()) + pre_blocks + 16
    perm = rng.permutation(num_blocks)
    prefix_ids, perm = perm[:pre_blocks], perm[pre_blocks:]
    # each sequence's blocks, the new ones the lowest free ids in sequence order
    old, free = perm[:int(held.sum())], np.sort(perm[int(held.sum()):])
    before, table = np.full((S, MB), -1), np.full((S, MB), -1)
    a = b = 0
    for s in range(S):
        before[s, :held[s]] = old[a:a + held[s]]
        table[s, :held[s]] = before[s, :held[s]]
        table[s, held[s]:need[s]] = free[b:b + need[s] - held[s]]
        a, b = a + held[s], b + need[s] - held[s]
    bits = np.zeros(-(-num_blocks // 32) * 32, np.uint8)
    bits[free] = 1

    def words(x):
        w = np.packbits(x, bitorder="little").view("<u4").astype(np.int64)
        return _int32(np.where(w >= 2 ** 31, w - 2 ** 32, w))

    free_before = words(bits)
    bits[free[:b]] = 0
    capacity = max(1, int(n_new.sum()) + c["pad"])
    if c["op"] != "rotary":
        capacity = c["decodes"] * c["nodes"] + c["prompts"] * c["rows"] + c["pad"]
    q_start = np.concatenate([[0], np.cumsum(n_new)])
    parent, position, slot = (np.full(capacity, -1) for _ in range(3))
    token, chosen = (rng.integers(1000, 30000, capacity) for _ in range(2))
    given = np.where(n_new > 0, np.where(drafted, 1, n_new), 0)
    seq = np.zeros(capacity, np.int64)
    depth = 1
    for s in range(S):
        n, q0 = int(n_new[s]), int(q_start[s])
        if n == 0:
            continue
        mine = _parents(n, int(rng.integers(1, 5)) if drafted[s] else 1)
        parent[q0:q0 + n] = mine
        pos = seen[s] + np.arange(n)
        position[q0:q0 + n] = pos
        slot[q0:q0 + n] = table[s, pos // B] * B + pos % B
        seq[q0:q0 + n] = s
        # siblings' tokens differ; the tokens chosen lead along a path and then off the tree
        token[q0:q0 + n] = 1000 + 10 * np.arange(n) + s % 7
        chosen[q0:q0 + n] = 5
        if drafted[s]:
            path = _path(mine, rng)
            chosen[q0 + np.array(path[:-1], np.int64)] = token[q0 + np.array(path[1:], np.int64)]
        else:
            chosen[q0:q0 + n - 1] = token[q0 + 1:q0 + n]
        if n <= _MAX_NODES:
            depth = max(depth, n if mine[-1] == n - 2 else 32)
    s = {"case": c, "capacity": capacity, "num_blocks": num_blocks, "depth": depth,
         "seen": _int32(seen), "n_new": _int32(n_new), "table": _int32(table),
         "free": words(bits), "q_start": _int32(q_start), "parent": _int32(parent),
         "position": _int32(position), "slot": _int32(slot), "token": _int32(token),
         "chosen": _int32(chosen), "given": _int32(given), "seq": torch.from_numpy(seq).cuda(),
         "lengths": (seen.tolist(), n_new.tolist(), q_start.tolist()),
         "longest_new": int(n_new.max())}
    if own:
        import ragged_blocked_kv_gb300 as rbkv
        cfg = rbkv.Config(c["hq"], c["hkv"], c["dim"], B, c["dtype"], num_blocks)
        t = s["tables"] = rbkv.StepTables(cfg, S, MB, capacity)
        t.build(s["seen"], s["n_new"], block_table=_int32(before), free=free_before)
        if c["op"] == "rotary":
            s["rotary"] = rbkv.Rotary(c["rot"], base=c["base"], layout=c["layout"],
                                      scaling=c["scaling"], factor=c["factor"],
                                      original_length=8192, low=1.0, high=32.0)
        else:
            s["draft"] = rbkv.StepDraft(t)
            s["draft"].plan(s["parent"])
    if c["op"] == "draft":
        return s
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    dt = _DTYPES[c["dtype"]]

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda", dtype=torch.float32).to(dt)

    cache = (num_blocks, c["hkv"], B, c["dim"])
    s["k_cache"], s["v_cache"] = normal(*cache), normal(*cache)
    if c["op"] == "accept":
        return s
    s["q"] = normal(capacity, c["hq"], c["dim"])
    s["o"] = torch.zeros_like(s["q"])
    if c["op"] == "rotary":
        s["k_new"], s["v_new"] = (normal(capacity, c["hkv"], c["dim"]) for _ in range(2))
        s["inv_freq"] = torch.from_numpy(_inv_freq(c)).cuda()
        return s
    s["prefix"] = _int32(prefix_ids)
    s["sets"] = _ancestors(s)[0]
    if own:
        s["workspace"] = torch.empty(max(256, s["tables"].workspace_bytes(c["prefix"])),
                                     dtype=torch.uint8, device="cuda")
    return s


# ---- plain forms -------------------------------------------------------------------
def _rotate(x, cos, sin, c):
    """x [rows][heads][dim] in 32 bits, cos and sin [rows][rot / 2]."""
    R = c["rot"]
    cos, sin = cos[:, None], sin[:, None]
    out = x.clone()
    if c["layout"] == "half":
        a, b = slice(0, R // 2), slice(R // 2, R)
    else:
        a, b = slice(0, R, 2), slice(1, R, 2)
    out[..., a] = x[..., a] * cos - x[..., b] * sin
    out[..., b] = x[..., b] * cos + x[..., a] * sin
    return out


def _rotary_plain(s):
    c, B = s["case"], s["case"]["block"]
    live = s["position"] >= 0
    T = s["lengths"][2][-1]
    angle = (s["position"][:T].double() + c["prefix"])[:, None] * s["inv_freq"]
    cos, sin = torch.cos(angle).float(), torch.sin(angle).float()
    dt, slot = s["q"].dtype, s["slot"][:T].long()
    q = s["o"].clone()
    q[:T] = _rotate(s["q"][:T].float(), cos, sin, c).to(dt)
    k = _rotate(s["k_new"][:T].float(), cos, sin, c).to(dt)
    s["k_cache"][slot // B, :, slot % B] = k
    s["v_cache"][slot // B, :, slot % B] = s["v_new"][:T]
    return {"q": torch.where(live[:, None, None], q, s["o"]), "k_cache": s["k_cache"],
            "v_cache": s["v_cache"]}


def _ancestors(s):
    """One truth value per row and token of its tree: itself and what it follows."""
    T, dev = s["capacity"], s["parent"].device
    live = s["position"] >= 0
    q0 = s["q_start"].long()[s["seq"]]
    index = torch.arange(T, device=dev) - q0
    short = live & (s["n_new"].long()[s["seq"]] <= _MAX_NODES)
    seen = torch.zeros(T, _MAX_NODES + 1, dtype=torch.bool, device=dev)
    node = torch.where(short, index, -1)
    row, parent = torch.arange(T, device=dev), s["parent"].long()
    for _ in range(s["depth"]):
        seen[row, torch.where(node >= 0, node, _MAX_NODES)] = True
        node = torch.where(node >= 0, parent[(q0 + node).clamp(0, T - 1)], -1)
    return seen[:, :_MAX_NODES], index, short, live


def _draft_plain(s):
    seen, index, short, live = _ancestors(s)
    start = s["seen"].long()[s["seq"]]
    place = torch.where(live, start + torch.where(short, seen.sum(1) - 1, index), -1)
    word = (seen.reshape(-1, 4, 32).long() << torch.arange(32, device=seen.device)).sum(-1)
    word = torch.where(word >= 2 ** 31, word - 2 ** 32, word)
    return {"place": place.to(torch.int32), "ancestors": word.to(torch.int32)}


def _keys(cache, ids, n):
    """The first n rows of a block list: [kv heads, n, dim] in 32 bits."""
    B = cache.shape[2]
    x = cache[ids[:-(-n // B)].long()].transpose(1, 2).reshape(-1, *cache.shape[1::2])
    return x[:n].transpose(0, 1).float()


def _tree_plain(s):
    c = s["case"]
    hkv, g, dim, P = c["hkv"], c["hq"] // c["hkv"], c["dim"], c["prefix"]
    sets = s["sets"]
    seen, n_new, q_start = s["lengths"]
    k_pre, v_pre = (_keys(x, s["prefix"], P) for x in (s["k_cache"], s["v_cache"]))
    out = s["o"].clone()
    for i, (before, n, row) in enumerate(zip(seen, n_new, q_start)):
        if n == 0:
            continue
        k, v = (torch.cat([pre, _keys(x, s["table"][i], before + n)], 1)
                for pre, x in ((k_pre, s["k_cache"]), (v_pre, s["v_cache"])))
        q = s["q"][row:row + n].float().reshape(n, hkv, g, dim).permute(1, 2, 0, 3)
        score = torch.matmul(q.reshape(hkv, g * n, dim) * dim ** -0.5, k.transpose(1, 2))
        score = score.reshape(hkv, g, n, P + before + n)
        if n <= _MAX_NODES:
            sees = sets[row:row + n, :n]
        else:
            sees = torch.ones(n, n, dtype=torch.bool, device=q.device).tril()
        score[..., P + before:] = torch.where(sees, score[..., P + before:], float("-inf"))
        weight = torch.exp(score - score.amax(-1, keepdim=True))
        total = weight.sum(-1, keepdim=True)
        o = torch.matmul(weight.reshape(hkv, g * n, -1), v).reshape(hkv, g, n, dim) / total
        out[row:row + n] = o.permute(2, 0, 1, 3).reshape(n, hkv * g, dim).to(out.dtype)
    return out


def _accept_plain(s):
    c, B = s["case"], s["case"]["block"]
    S, N, dev = len(s["seen"]), s["longest_new"], s["seen"].device
    col = torch.arange(N, device=dev)
    q0, n_new, given = s["q_start"].long()[:-1], s["n_new"].long(), s["given"].long()
    inside = col < n_new[:, None]
    row = (q0[:, None] + col).clamp(max=s["capacity"] - 1)
    parent = torch.where(inside, s["parent"].long()[row], -2)
    token, chosen = s["token"].long()[row], s["chosen"].long()[row]
    path = torch.where(col < given[:, None], col, -1)
    count, cur = given.clone(), (given - 1).clamp(min=0)
    for _ in range(min(s["depth"], N)):
        want = chosen.gather(1, cur[:, None])
        match = (parent == cur[:, None]) & (token == want) & (col > cur[:, None])
        found = match.any(1) & (n_new > 0)
        child = match.to(torch.int8).argmax(1)
        at = torch.where(found, count, N)
        path = torch.nn.functional.pad(path, (0, 1))
        path.scatter_(1, at[:, None], torch.where(found, child, -1)[:, None])
        path = path[:, :N]
        count, cur = count + found, torch.where(found, child, cur)
    busy = n_new > 0
    kept = (col < count[:, None]) & inside
    rows = torch.full((s["capacity"] + 1,), -1, dtype=torch.long, device=dev)
    rows.scatter_(0, torch.where(kept, q0[:, None] + col, s["capacity"]).reshape(-1),
                  torch.where(kept, q0[:, None] + path, -1).reshape(-1))
    rows = rows[:-1]
    ctx = s["seen"].long() + torch.where(busy, count, 0)
    # blocks past the kept tokens
    block = torch.arange(s["table"].shape[1], device=dev)
    gone = ((block >= ((ctx + B - 1) // B)[:, None]) &
            (block < ((s["seen"].long() + n_new + B - 1) // B)[:, None]))
    bits = ((s["free"].long()[:, None] >> torch.arange(32, device=dev)) & 1).reshape(-1)
    bits = torch.cat([bits, bits[:1]])
    bits.scatter_(0, torch.where(gone, s["table"].long(), len(bits) - 1).reshape(-1),
                  torch.ones(gone.numel(), dtype=torch.long, device=dev))
    word = (bits[:-1].reshape(-1, 32) << torch.arange(32, device=dev)).sum(1)
    free = torch.where(word >= 2 ** 31, word - 2 ** 32, word)
    # the kept rows, together
    T = s["lengths"][2][-1]
    slot = s["slot"].long()
    to = slot[:T]
    source = torch.where(rows[:T] >= 0, slot[rows[:T].clamp(min=0)], to)
    for x in (s["k_cache"], s["v_cache"]):
        x[to // B, :, to % B] = x[source // B, :, source % B]
    last = chosen.gather(1, cur[:, None])[:, 0]
    out = {"path": rows, "accepted": torch.where(busy, count, 0),
           "next_token": torch.where(busy, last, -1), "ctx": ctx, "free": free}
    out = {k: v.to(torch.int32) for k, v in out.items()}
    return {**out, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def run(state):
    s, c, op = state, state["case"], state["case"]["op"]
    if not own:
        return {"rotary": _rotary_plain, "draft": _draft_plain, "tree": _tree_plain,
                "accept": _accept_plain}[op](s)
    t, d = s["tables"], s.get("draft")
    if op == "rotary":
        q = t.append_rotary(s["rotary"], s["q"], s["k_new"], s["v_new"], s["k_cache"],
                            s["v_cache"], q_out=s["o"], prefix_len=c["prefix"])
        return {"q": q, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}
    if op == "draft":
        d.plan(s["parent"])
        return {"place": d.place, "ancestors": d.ancestors}
    if op == "tree":
        return t.attention(s["q"], s["k_cache"], s["v_cache"], prefix_table=s["prefix"],
                           prefix_len=c["prefix"], o=s["o"], workspace=s["workspace"], draft=d)
    d.accept(s["token"], s["chosen"], s["given"])
    d.compact(s["k_cache"], s["v_cache"])
    return {"path": d.path, "accepted": d.accepted, "next_token": d.next_token, "ctx": t.ctx,
            "free": t.free, "k_cache": s["k_cache"], "v_cache": s["v_cache"]}


def work(case):
    """One pass at the mean lengths of the case's distribution."""
    c, op = case, case["op"]
    each = 1 if op == "rotary" else ((c["nodes"] + 1) // 2 + c["nodes"]) / 2
    T = c["decodes"] * each + c["prompts"] * c["rows"]
    size = 2 if c["dtype"] == "bf16" else 4
    row = c["dim"] * size
    if op == "rotary":
        return {"bytes": int(2 * T * (c["hq"] + 2 * c["hkv"]) * row + 8 * T),
                "flops": int(3 * T * (c["hq"] + c["hkv"]) * c["rot"])}
    if op == "draft":
        return {"bytes": int(24 * T), "flops": int(4 * T)}
    if op == "accept":
        moved = c["decodes"] * math.log2(1 + each) / 2
        return {"bytes": int(32 * T + 4 * moved * c["hkv"] * row), "flops": int(T)}
    mean = (c["own_lo"] + c["own_hi"]) / 2
    keys = c["decodes"] * (mean + each) + c["prompts"] * (20 + c["rows"])
    pairs = (c["decodes"] * each * (c["prefix"] + mean + math.log2(1 + each)) +
             c["prompts"] * c["rows"] * (c["prefix"] + 20 + c["rows"] / 2))
    return {"bytes": int((2 * (c["prefix"] + keys) * c["hkv"] + 2 * T * c["hq"]) * row),
            "flops": int(4 * c["dim"] * c["hq"] * pairs)}


# ---- in 64 bits, from the definitions -----------------------------------------------
def exact(case, seed):
    """Rotations by complex factors; attention by sequence, every token's keys looked up by
    walking its tree.  The other operators' outputs are whole numbers and copies."""
    if case["op"] not in ("rotary", "tree"):
        return None
    c, s = case, prepare(case, seed)
    dim, B = c["dim"], c["block"]
    seen, n_new, q_start = s["lengths"]
    if c["op"] == "rotary":
        R, T = c["rot"], q_start[-1]
        turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"),
                           (s["position"][:T].double() + c["prefix"])[:, None, None] *
                           torch.from_numpy(_inv_freq(c)).cuda())

        def rotated(x):
            x = x.double()
            head = x[..., :R]
            pairs = head.unflatten(-1, (2, R // 2)).transpose(-1, -2) if c["layout"] == "half" \
                else head.unflatten(-1, (R // 2, 2))
            y = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn)
            y = y.transpose(-1, -2) if c["layout"] == "half" else y
            return torch.cat([y.flatten(-2), x[..., R:]], -1)

        q, k_cache = s["o"].double(), s["k_cache"].double()
        q[:T] = rotated(s["q"][:T])
        for r, (row, at) in enumerate(zip(rotated(s["k_new"][:T]), s["slot"][:T].tolist())):
            k_cache[at // B, :, at % B] = row
        return {"q": q, "k_cache": k_cache, "v_cache": None}
    g, P = c["hq"] // c["hkv"], c["prefix"]
    parent, table = s["parent"].cpu().numpy(), s["table"].cpu().numpy()
    prefix = s["prefix"].cpu().numpy()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    for i, (before, n, row) in enumerate(zip(seen, n_new, q_start)):
        if n == 0:
            continue
        p = np.arange(P)
        o = np.arange(before + n)
        where = np.concatenate([prefix[p // B] * B + p % B, table[i, o // B] * B + o % B])
        where = torch.from_numpy(where.astype(np.int64)).cuda()
        k, v = (x[where // B, :, where % B].double().permute(1, 0, 2)
                for x in (s["k_cache"], s["v_cache"]))
        hidden = np.ones((n, P + before + n), bool)
        hidden[:, :P + before] = False
        for r in range(n):
            node = r
            while node >= 0:
                hidden[r, P + before + node] = False
                node = int(parent[row + node])
        hidden = torch.from_numpy(hidden).cuda()
        for h in range(c["hkv"]):
            q = s["q"][row:row + n, h * g:(h + 1) * g].double().transpose(0, 1)
            logit = (q @ k[h].T / dim ** 0.5).masked_fill(hidden, float("-inf"))
            out[row:row + n, h * g:(h + 1) * g] = (torch.softmax(logit, -1) @ v[h]).transpose(0, 1)
    return out
