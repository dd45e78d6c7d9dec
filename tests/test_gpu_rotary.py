"""Appends with a rotation on the way: steps, passes and frames against the oracle."""
import numpy as np
import pytest
import torch

import oracle
import workloads
from draft_harness import random_trees, rotary_bound
from step_harness import i32
from test_gpu_step import BOUNDS, INVALID, MIXED, _case

pytestmark = pytest.mark.gpu

# heads, KV heads, head dim, block, type; rotated elements
SHAPES = [((8, 2, 64, 16, "f32"), 64), ((4, 4, 32, 5, "f32"), 8), ((3, 1, 256, 16, "f32"), 256),
          ((8, 2, 64, 16, "bf16"), 16), ((6, 2, 96, 24, "bf16"), 24), ((6, 2, 96, 24, "bf16"), 96),
          ((32, 8, 128, 64, "bf16"), 128), ((32, 32, 128, 64, "bf16"), 64),
          ((64, 1, 128, 16, "bf16"), 20), ((5, 5, 32, 7, "f32"), 2), ((10, 2, 160, 32, "bf16"), 80),
          ((8, 8, 64, 16, "f32"), 20), ((8, 8, 64, 16, "f32"), 22), ((8, 2, 64, 16, "bf16"), 6),
          ((4, 1, 128, 8, "bf16"), 40), ((4, 1, 128, 8, "bf16"), 124)]


def _rope(rbkv, R, layout, **kw):
    return rbkv.Rotary(R, base=kw.pop("base", 500.0), layout=layout, **kw)


def _rows(T, shape, seed=1):
    hq, hkv, D, _, dtype = shape
    gen = torch.Generator().manual_seed(seed)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    return [torch.randn(T, h, D, generator=gen).to(dt) for h in (hq, hkv, hkv)]


def _close(got, x, position, rope, dtype):
    exact = oracle.draft.rotate(x.double().numpy(), position, rope.inv_freq, rope.layout,
                                np.float32(rope.scale))
    bound = rotary_bound(x.double().numpy(), position, rope.inv_freq, rope.layout,
                         np.float32(rope.scale), exact, dtype)
    err = np.abs(got.double().cpu().numpy() - exact)
    assert (err <= bound).all(), float((err / bound).max())


def _check_step(t, want, rope, tensors, caches, before, q_out, old, prefix, position, shape):
    """q_out, the caches' new rows and everything that had to stay."""
    q, k, v = tensors
    B, dtype, rows = shape[3], shape[4], int(want.q_start[-1])
    place = np.asarray(position[:rows]) + prefix
    _close(q_out[:rows], q[:rows], place, rope, dtype)
    assert torch.equal(q_out[rows:].cpu(), old[rows:])
    slot = torch.from_numpy(want.slot[:rows].astype(np.int64))
    kc, vc = (c.cpu() for c in caches)
    _close(kc[slot // B, :, slot % B], k[:rows], place, rope, dtype)
    for c, b in ((kc, before[0].clone()), (vc, before[1].clone())):
        b[slot // B, :, slot % B] = v[:rows] if c is vc else c[slot // B, :, slot % B]
        assert torch.equal(c, b)


@pytest.mark.parametrize("shape,R", SHAPES, ids=str)
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("in_place", [False, True])
def test_step_against_oracle(rbkv, shape, R, layout, in_place):
    t, want, _, kd, vd, kc, vc, *_ = _case(rbkv, *shape, 0, *MIXED, pad=5)
    q, k, v = _rows(t.max_tokens, shape)
    rope = _rope(rbkv, R, layout, scale=1.25)
    qd = q.cuda()
    out = qd if in_place else torch.full_like(qd, 7.0)
    old = out.cpu().clone()
    assert t.append_rotary(rope, qd, k.cuda(), v.cuda(), kd, vd, q_out=out, prefix_len=1000) is out
    t.device_status()
    _check_step(t, want, rope, (q, k, v), (kd, vd), (kc, vc), out, old, 1000, want.position, shape)
    assert in_place or torch.equal(qd.cpu(), q)


@pytest.mark.parametrize("prefix", [1, 2 ** 20 + 1, 2 ** 30])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_far_positions(rbkv, prefix, layout):
    """Angles of a billion turns: what a 32-bit product would lose."""
    shape = (8, 2, 64, 16, "f32")
    t, want, _, kd, vd, kc, vc, *_ = _case(rbkv, *shape, 0, *MIXED)
    q, k, v = _rows(t.max_tokens, shape, 2)
    rope = rbkv.Rotary(64, layout=layout)
    out = t.append_rotary(rope, q.cuda(), k.cuda(), v.cuda(), kd, vd, prefix_len=prefix)
    _check_step(t, want, rope, (q, k, v), (kd, vd), (kc, vc), out, out.cpu(), prefix,
                want.position, shape)


@pytest.mark.parametrize("scaling", ["linear", "base", "parts"])
def test_scaled_and_given_angles(rbkv, scaling):
    shape = (32, 8, 128, 64, "bf16")
    t, want, _, kd, vd, kc, vc, *_ = _case(rbkv, *shape, 0, *MIXED)
    q, k, v = _rows(t.max_tokens, shape, 3)
    rope = rbkv.Rotary(128, scaling=scaling, factor=8.0, original_length=4096, scale=0.5)
    given = rbkv.Rotary(128, inv_freq=rope.inv_freq, scale=0.5)
    assert torch.equal(rope.turns, given.turns)
    out = t.append_rotary(given, q.cuda(), k.cuda(), v.cuda(), kd, vd, prefix_len=30000)
    _check_step(t, want, rope, (q, k, v), (kd, vd), (kc, vc), out, out.cpu(), 30000,
                want.position, shape)


@pytest.mark.parametrize("shape,R", [((32, 8, 128, 64, "bf16"), 128), ((8, 2, 64, 16, "f32"), 20)],
                         ids=str)
def test_drafted_tokens_turn_by_their_place(rbkv, shape, R):
    t, want, _, kd, vd, kc, vc, *_ = _case(rbkv, *shape, 0, *MIXED, pad=2)
    q, k, v = _rows(t.max_tokens, shape, 4)
    d = rbkv.StepDraft(t)
    parent = random_trees(np.random.default_rng(5), MIXED[1], t.max_tokens)
    out = torch.full_like(q, 7.0, device="cuda")
    rope = _rope(rbkv, R, "half")
    args = (rope, q.cuda(), k.cuda(), v.cuda(), kd, vd)
    t.append_rotary(*args, q_out=out, draft=d)          # not planned: nothing happens
    with pytest.raises(rbkv.RbkvError) as e:
        t.device_status()
    assert e.value.status == INVALID
    assert (out == 7.0).all() and torch.equal(kd.cpu(), kc) and torch.equal(vd.cpu(), vc)
    d.plan(i32(parent))
    t.append_rotary(*args, q_out=out, prefix_len=9, draft=d)
    t.device_status()
    plan = oracle.draft.plan(want, parent, t.max_tokens)
    assert plan.good
    _check_step(t, want, rope, (q, k, v), (kd, vd), (kc, vc), out, torch.full_like(q, 7.0), 9,
                plan.place, shape)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("R", [64, 20])
def test_what_is_not_rotated_is_copied(rbkv, dtype, R):
    """Infinities and NaN behind the rotated elements, in values, and in another pair;
    the bits of NaN, too."""
    shape = (4, 2, 96, 8, dtype)
    t, want, _, kd, vd, kc, vc, *_ = _case(rbkv, *shape, 0, [3, 0], [2, 9])
    q, k, v = _rows(t.max_tokens, shape, 5)
    q[0, 1, R], q[1, 2, R + 1], q[2, 0, 95] = float("inf"), float("nan"), float("-inf")
    k[3, 1, 95], k[0, 0, 5], v[4, 0, 7] = float("nan"), float("inf"), float("nan")
    rope = _rope(rbkv, R, "half")
    out = t.append_rotary(rope, q.cuda(), k.cuda(), v.cuda(), kd, vd).cpu()
    raw = torch.int16 if dtype == "bf16" else torch.int32
    assert torch.equal(out[..., R:].contiguous().view(raw), q[..., R:].contiguous().view(raw))
    slot = torch.from_numpy(want.slot.astype(np.int64))
    new_v, new_k = vd.cpu()[slot // 8, :, slot % 8], kd.cpu()[slot // 8, :, slot % 8]
    assert torch.equal(new_v.contiguous().view(raw), v.view(raw))
    bad = ~torch.isfinite(new_k)
    assert bad[3, 1, 95] and bad[0, 0, 5] and bad[0, 0, 5 + R // 2] and bad.sum() == 3
    assert torch.isfinite(out[..., :R]).all()


def test_bad_slots_and_another_configuration(rbkv):
    shape = (8, 2, 64, 16, "f32")
    t, want, _, kd, vd, kc, vc, *_ = _case(rbkv, *shape, 0, [40, 3], [1, 2])
    q, k, v = _rows(t.max_tokens, shape, 6)
    t.slot[1] = -1                                       # (as a table with a bad id makes it)
    rope = _rope(rbkv, 64, "half")
    out = t.append_rotary(rope, q.cuda(), k.cuda(), v.cuda(), kd, vd)
    with pytest.raises(rbkv.RbkvError) as e:
        t.device_status()
    assert e.value.status == BOUNDS
    _close(out, q, want.position, rope, "f32")           # (the queries need no slot)
    slot = [int(want.slot[0]), int(want.slot[2])]
    _close(torch.stack([kd[s // 16, :, s % 16] for s in slot]), k[[0, 2]], want.position[[0, 2]],
           rope, "f32")
    for s in slot:
        kc[s // 16, :, s % 16] = kd[s // 16, :, s % 16].cpu()
    assert torch.equal(kd.cpu(), kc)
    # built for another block size
    other = rbkv.StepTables(rbkv.Config(8, 2, 64, 8, "f32", 2 * t.config.num_blocks), 2,
                            t.max_blocks, t.max_tokens)
    other.plan.copy_(t.plan)
    out = torch.full_like(q, 7.0, device="cuda")
    other.append_rotary(rope, q.cuda(), k.cuda(), v.cuda(), kd.view(-1, 2, 8, 64),
                        vd.view(-1, 2, 8, 64), q_out=out)
    with pytest.raises(rbkv.RbkvError) as e:
        other.device_status()
    assert e.value.status == INVALID and (out == 7.0).all()


def test_captured_on_a_side_stream(rbkv):
    """build and append of a decoding loop, captured, replayed twice; without q_out."""
    shape, side = (32, 8, 128, 64, "bf16"), torch.cuda.Stream()
    cfg = rbkv.Config(*shape, 40)
    t = rbkv.StepTables(cfg, 3, 4, 3)
    kd, vd = (torch.zeros(cfg.cache_shape(), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    q, k, v = (x.cuda() for x in _rows(3, shape, 7))
    rope, one = _rope(rbkv, 128, "interleaved"), torch.ones(3, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()

    def step(**kw):
        t.build(t.ctx, one, **kw)
        return t.append_rotary(rope, q, k, v, kd, vd, prefix_len=50, **kw)

    out = step(stream=side)
    side.synchronize()
    _close(out, q.cpu(), [50] * 3, rope, "bf16")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in (1, 2):
        graph.replay()
        torch.cuda.synchronize()
        _close(out, q.cpu(), [50 + i] * 3, rope, "bf16")
    for s in range(3):
        blk = int(t.block_table[s, 0])
        for i in range(3):
            _close(kd[blk, :, i][None], k[s:s + 1].cpu(), [50 + i], rope, "bf16")
            assert torch.equal(vd[blk, :, i], v[s])


@pytest.mark.parametrize("dtype,R", [("bf16", 128), ("bf16", 40), ("f32", 64)])
def test_pass_and_frame(rbkv, dtype, R):
    """A pass of a prompt chunk behind cached tokens, a fresh prompt and decodes; a frame
    gives the same bits."""
    shape = (8, 2, 128, 16, dtype)
    cfg = rbkv.Config(*shape, 64)
    comp = rbkv.Composer(cfg)
    dt = cfg.torch_dtype
    caches = [torch.zeros(cfg.cache_shape(), dtype=dt, device="cuda") for _ in range(4)]
    rope = _rope(rbkv, R, "half")
    for i, states in enumerate(([(1, 100, 0), (2, 9, 0)], [(1, 100, 70), (3, 33, 0), (2, 9, 9)])):
        p = comp.compose(79 if i == 0 else 200, 70, states)
        m = p.meta
        position = np.concatenate([s + np.arange(n) for s, n in zip(m.seen, m.n_new)])
        q, k, v = _rows(p.num_tokens, shape, i)
        frame = None
        if dtype == "bf16":
            frame = rbkv.Frame(cfg, p.num_tokens + 11, packed_units=1)
            p.set_chunk_items(frame.chunk_items)
        out = rbkv.kv_append_rotary(p, rope, q.cuda(), k.cuda(), v.cuda(), caches[0], caches[1])
        _close(out, q, position, rope, dtype)
        slot = torch.from_numpy(m.slot.astype(np.int64))
        _close(caches[0].cpu()[slot // 16, :, slot % 16], k, position, rope, dtype)
        assert torch.equal(caches[1].cpu()[slot // 16, :, slot % 16], v)
        p.device_status()
        if frame is not None:
            T = p.num_tokens
            frame.load(p)
            pad = [torch.full((T + 11, *x.shape[1:]), 5.0, dtype=dt, device="cuda")
                   for x in (q, k, v)]
            for x, y in zip(pad, (q, k, v)):
                x[:T] = y.cuda()
            mine = torch.full_like(pad[0], 7.0)
            frame.kv_append_rotary(rope, *pad, caches[2], caches[3], q_out=mine)
            frame.device_status()
            assert torch.equal(mine[:T], out) and (mine[T:] == 7.0).all()
            assert torch.equal(caches[0], caches[2]) and torch.equal(caches[1], caches[3])
    empty = comp.compose(0, 0, [])
    none = torch.empty(0, 8, 128, dtype=dt, device="cuda")
    kv = torch.empty(0, 2, 128, dtype=dt, device="cuda")
    assert rbkv.kv_append_rotary(empty, rope, none, kv, kv, caches[0], caches[1]).shape[0] == 0


def test_rotated_attention_goes_by_distance(rbkv):
    """A whole step, rotated: attention against fp64 over the exactly rotated rows, with
    what the roundings of q and k cost added to the bound (2^-8 of each, so 2^-7 of a
    score's sum of magnitudes, twice: once for the weights' sum)."""
    from step_harness import error_bound, reference
    shape, P = (16, 4, 128, 64, "bf16"), 0
    n_new = MIXED[1]
    t, want, _, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, P, [0] * len(n_new), n_new)
    q, k, v = _rows(t.max_tokens, shape, 8)
    rope = _rope(rbkv, 128, "half", base=10000.0)
    out = t.append_rotary(rope, q.cuda(), k.cuda(), v.cuda(), kd, vd)
    o = t.attention(out, kd, vd).cpu()[:rows].double()
    t.device_status()
    kx, vx = kc.double(), vc.double()
    turned = torch.from_numpy(oracle.draft.rotate(k.double().numpy(), np.maximum(want.position, 0),
                                                  rope.inv_freq, "half"))
    for r in range(rows):
        b, off = divmod(int(want.slot[r]), 64)
        kx[b, :, off], vx[b, :, off] = turned[r], v[r].double()
    qx = torch.from_numpy(oracle.draft.rotate(q.double().numpy(), np.maximum(want.position, 0),
                                              rope.inv_freq, "half"))
    ref = reference(want, qx, kx, vx, ids, P)
    slack = torch.expm1(2 * 2.0 ** -7 * 1.01 * ref[2]) * ref[1]
    err = (o - ref[0]).abs()
    assert (err <= error_bound(ref, 128, "bf16") + slack).all()


def test_layer_with_rotary_positions(rbkv):
    """DecoderLayer(rotary=...): its attention is that of rotated queries and keys."""
    from ragged_blocked_kv_gb300.layer import DecoderLayer, random_weights
    hidden, hq, hkv, D, ffn = 512, 4, 2, 128, 512
    w = random_weights(hidden, hq, hkv, D, ffn, seed=1)
    rope = rbkv.Rotary(128)
    cfg = rbkv.Config(hq, hkv, D, 64, "bf16", 16)
    outs = []
    for rotary in (None, rope):
        comp = rbkv.Composer(cfg)
        kc, vc = (torch.zeros(cfg.cache_shape(), dtype=torch.bfloat16, device="cuda")
                  for _ in range(2))
        layer = DecoderLayer(rbkv, w, hq, hkv, D, rotary=rotary)
        p = comp.compose(300, 0, [(1, 200, 0), (2, 5, 0)])
        x = torch.randn(205, hidden, generator=torch.Generator().manual_seed(3)).to(torch.bfloat16)
        outs.append(layer.forward(p, x.cuda(), kc, vc))
        m = p.meta
        slot = torch.from_numpy(m.slot.astype(np.int64))
        outs[-1]["cached"] = kc.cpu()[slot // 64, :, slot % 64]
    plain, turned = outs
    position = np.concatenate([np.arange(200), np.arange(5)])
    assert torch.equal(plain["cached"], plain["k"].cpu())
    assert torch.equal(turned["k"], plain["k"])
    _close(turned["q"], plain["q"].cpu(), position, rope, "bf16")
    _close(turned["cached"], plain["k"].cpu(), position, rope, "bf16")
    first = [0, 200]                                     # one key: position changes nothing
    assert torch.equal(plain["out"][first], turned["out"][first])
    assert not torch.equal(plain["out"][100], turned["out"][100])


def test_offsets_past_two_to_the_31(rbkv):
    """Slots whose rows lie behind 2^31 elements."""
    shape = (8, 8, 128, 64, "bf16")
    blocks = 33000                                       # 33000 * 65536 elements
    cfg = rbkv.Config(*shape, blocks)
    t = rbkv.StepTables(cfg, 2, 4, 4)
    t.free.zero_()
    t.free[(blocks - 1) // 32] = 1 << ((blocks - 1) % 32)
    t.free[1] = 1
    t.build(t.ctx, i32([2, 1]))
    assert t.block_table[:, 0].tolist() == [32, blocks - 1]
    kd, vd = (torch.zeros(cfg.cache_shape(), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    q, k, v = _rows(4, shape, 9)
    rope = _rope(rbkv, 128, "half")
    t.append_rotary(rope, q.cuda(), k.cuda(), v.cuda(), kd, vd)
    t.device_status()
    assert torch.equal(vd[blocks - 1, :, 0].cpu(), v[2])
    _close(kd[blocks - 1, :, 0][None], k[2:3], [0], rope, "bf16")
    assert not kd[blocks - 1, :, 1:].any() and torch.equal(vd[32, :, 1].cpu(), v[1])
