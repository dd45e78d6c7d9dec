"""Calls on steps as the interface allows them: at once on two streams, captured
across streams and beside copies, without a workspace, on shared blocks."""
import numpy as np
import pytest
import torch

from step_harness import error_bound, i32, reference
from test_gpu_step import MIXED, _case

pytestmark = pytest.mark.gpu

SHAPES = [(32, 8, 128, 64, "bf16"), (8, 2, 64, 16, "f32")]


def _good(o, ref, rows, shape):
    err = (o[:rows].cpu().double() - ref[0]).abs()
    return bool((err <= error_bound(ref, shape[2], shape[4])).all())


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_two_attentions_of_one_step_at_once(rbkv, shape):
    """Two layers' attention on one step's tables, on two streams, a workspace each."""
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 700, *MIXED)
    idc, sides, runs = i32(ids), [torch.cuda.Stream() for _ in range(2)], []
    for i in range(2):
        q2 = torch.randn(q.shape, generator=torch.Generator().manual_seed(i)).to(q.dtype)
        ws = torch.empty(max(256, t.workspace_bytes(700)), dtype=torch.uint8, device="cuda")
        runs.append((q2, q2.cuda(), torch.zeros_like(q2, device="cuda"), ws))
    torch.cuda.synchronize()
    for _ in range(10):
        for side, (_, qd, o, ws) in zip(sides, runs):
            t.attention(qd, kd, vd, prefix_table=idc, prefix_len=700, o=o, workspace=ws,
                        stream=side)
    torch.cuda.synchronize()
    t.device_status()
    for q2, _, o, _ in runs:
        assert _good(o, reference(want, q2, kc, vc, ids, 700), rows, shape)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_capture_across_streams_and_copies(rbkv, shape):
    """build - copies - append on a side stream - attention without a workspace
    or an output, beside a copy - release, as one graph, replayed on new inputs."""
    hq, hkv, D, B, dtype = shape
    t0, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 200, *MIXED, pad=4)
    cfg, T, S = t0.config, t0.max_tokens, t0.num_seqs
    t = rbkv.StepTables(cfg, S, t0.max_blocks, T)
    seen, new = i32(MIXED[0]), i32(MIXED[1])
    table, free = t0.block_table.clone(), t0.free.clone()   # (the step's blocks are taken here)
    held = -(-np.asarray(MIXED[0]) // B)
    for s in range(S):
        for c in range(held[s], -(-int(want.ctx[s]) // B)):
            b = int(want.table[s, c])
            free[b // 32] |= (1 << b % 32) if b % 32 < 31 else -2 ** 31
            table[s, c] = -1
    qin, kin, vin = (torch.zeros(T, h, D, dtype=q.dtype, device="cuda") for h in (hq, hkv, hkv))
    qd, kn, vn = (torch.empty_like(x) for x in (qin, kin, vin))
    idc, done, side = i32(ids), torch.ones(S, dtype=torch.int32, device="cuda"), torch.cuda.Stream()
    spare = torch.zeros(1 << 20, device="cuda")

    def step():
        t.build(seen, new, block_table=table, free=free)
        kn.copy_(kin)
        vn.copy_(vin)
        main = torch.cuda.current_stream()
        side.wait_stream(main)
        t.append(kn, vn, kd, vd, stream=side)
        qd.copy_(qin)
        main.wait_stream(side)
        o = t.attention(qd, kd, vd, prefix_table=idc, prefix_len=200)
        spare.zero_()
        t.release(done)
        return o

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = step()
    gen = torch.Generator().manual_seed(1)
    for _ in range(3):
        q2, k2, v2 = (torch.randn(T, h, D, generator=gen).to(q.dtype) for h in (hq, hkv, hkv))
        for x, y in ((qin, q2), (kin, k2), (vin, v2)):
            x.copy_(y)
        graph.replay()
        torch.cuda.synchronize()
        t.device_status()
        for r in range(rows):
            b, off = divmod(int(want.slot[r]), B)
            kc[b, :, off], vc[b, :, off] = k2[r], v2[r]
        assert _good(o, reference(want, q2, kc, vc, ids, 200), rows, shape)
        assert not t.ctx.any()


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_shared_blocks_and_one_cache_for_keys_and_values(rbkv, shape):
    """A prefix that lists a block twice and a sequence's own block; K = V."""
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 3 * shape[3], *MIXED)
    ids = np.array(ids)
    ids[1], ids[2] = ids[0], want.table[5, 0]
    P = 3 * shape[3] - 2
    o = t.attention(q.cuda(), kd, kd, prefix_table=i32(ids), prefix_len=P)
    t.device_status()
    assert _good(o, reference(want, q, kc, kc, ids, P), rows, shape)


@pytest.mark.parametrize("shape", SHAPES, ids=str)
def test_a_step_far_below_its_capacity(rbkv, shape):
    """Four live rows in tables of 300 sequences and 5000 rows."""
    S = 300
    seen, n_new = np.zeros(S, int), np.zeros(S, int)
    seen[[7, 120, 299]], n_new[[7, 120, 299]] = [100, 0, 700], [1, 2, 1]
    for prefix in (0, 2000):
        t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, prefix, seen, n_new, pad=4996)
        o = torch.full_like(q, 7.0, device="cuda")
        t.attention(q.cuda(), kd, vd, prefix_table=i32(ids) if prefix else None,
                    prefix_len=prefix, o=o)
        t.device_status()
        assert rows == 4 and (o[rows:] == 7.0).all()
        assert _good(o, reference(want, q, kc, vc, ids, prefix), rows, shape)


def test_layers_of_one_step_in_a_row(rbkv):
    """Append and attention of 24 layers behind one another, one workspace: each
    layer's result is its own."""
    shape, P = (16, 4, 128, 32, "bf16"), 150
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, P, *MIXED)
    gen, layers = torch.Generator().manual_seed(2), []
    ws = torch.empty(max(256, t.workspace_bytes(P)), dtype=torch.uint8, device="cuda")
    for _ in range(24):
        k, v, ql = kc.clone(), vc.clone(), torch.randn(q.shape, generator=gen).to(q.dtype)
        kn, vn = (torch.randn(t.max_tokens, 4, 128, generator=gen).to(q.dtype) for _ in range(2))
        layers.append([ql.cuda(), kn.cuda(), vn.cuda(), k.cuda(), v.cuda(), None, (ql, k, v, kn, vn)])
    torch.cuda.synchronize()
    for x in layers:
        t.append(x[1], x[2], x[3], x[4])
        x[5] = t.attention(x[0], x[3], x[4], prefix_table=i32(ids), prefix_len=P, workspace=ws)
    t.device_status()
    for *_, o, (ql, k, v, kn, vn) in layers[::5]:
        for r in range(rows):
            b, off = divmod(int(want.slot[r]), 32)
            k[b, :, off], v[b, :, off] = kn[r], vn[r]
        assert _good(o, reference(want, ql, k, v, ids, P), rows, shape)
