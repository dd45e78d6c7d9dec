"""Calls on a step with another configuration, or tables of other sizes, than
it was built for: nothing is written, and the status words say so.  Through the
C entries (a StepTables object has one configuration)."""
import ctypes as C

import numpy as np
import pytest
import torch

from step_harness import error_bound, i32, reference
from test_gpu_step import INVALID, MIXED, WORKSPACE, _case

pytestmark = pytest.mark.gpu


def _attention(rbkv, t, cfg, tables, q, k, v, ids, prefix, o, ws):
    L = rbkv.lib()
    return L.rbkv_step_attention(C.byref(cfg._c()), C.byref(tables), q.data_ptr(), k.data_ptr(),
                                 v.data_ptr(), ids.data_ptr(), prefix, o.data_ptr(),
                                 ws.data_ptr(), ws.nbytes, None)


def _refused(rbkv, t):
    with pytest.raises(rbkv.RbkvError) as e:
        t.device_status()
    assert e.value.status == INVALID


# (hq, hkv, D, block, dtype) of the build, and of the call
OTHERS = [((32, 8, 128, 64, "bf16"), (64, 8, 128, 64, "bf16")),     # a larger group
          ((32, 8, 128, 64, "bf16"), (8, 8, 128, 64, "bf16")),      # a smaller one
          ((32, 8, 128, 64, "bf16"), (32, 8, 128, 32, "bf16")),     # another block size
          ((32, 8, 128, 64, "bf16"), (8, 4, 64, 64, "f32")),        # another kernel
          ((8, 2, 64, 16, "f32"), (4, 2, 64, 16, "f32")),
          ((8, 2, 64, 16, "f32"), (8, 2, 64, 8, "f32"))]


@pytest.mark.parametrize("built,given", OTHERS, ids=str)
@pytest.mark.parametrize("batch", [MIXED, ([30], [1])], ids=["mixed", "one row"])
def test_attention_of_another_shape(rbkv, built, given, batch):
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *built, 200, *batch)
    hq, hkv, D, B, dtype = given
    cfg = rbkv.Config(hq, hkv, D, B, dtype, t.config.num_blocks)
    dt = cfg.torch_dtype
    caches = [torch.zeros(cfg.cache_shape(), dtype=dt, device="cuda") for _ in range(2)]
    qo = torch.zeros(t.max_tokens, hq, D, dtype=dt, device="cuda")
    o = torch.full_like(qo, 7.0)
    long_ids = torch.zeros(64, dtype=torch.int32, device="cuda")
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    assert _attention(rbkv, t, cfg, t._tables, qo, *caches, long_ids, 200, o, ws) == 0
    _refused(rbkv, t)
    assert (o == 7.0).all()
    # the step itself is as it was
    o = t.attention(q.cuda(), kd, vd, prefix_table=i32(ids), prefix_len=200)
    t.device_status()
    ref = reference(want, q, kc, vc, ids, 200)
    assert ((o[:rows].cpu().double() - ref[0]).abs() <= error_bound(ref, built[2], built[4])).all()


def test_the_same_group_with_other_heads(rbkv):
    """KV heads, head dim and type may differ from the build's."""
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, 32, 8, 128, 64, "bf16", 200, *MIXED)
    for hq, hkv, D, dtype in ((8, 2, 128, "bf16"), (4, 1, 64, "f32")):
        cfg = rbkv.Config(hq, hkv, D, 64, dtype, t.config.num_blocks)
        dt = cfg.torch_dtype
        k, v, q2 = (torch.randn(*s).to(dt) for s in (cfg.cache_shape(), cfg.cache_shape(),
                                                     (t.max_tokens, hq, D)))
        o = torch.zeros_like(q2, device="cuda")
        ws = torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
        kv, qc = (k.cuda(), v.cuda()), q2.cuda()
        assert _attention(rbkv, t, cfg, t._tables, qc, *kv, i32(ids), 200, o, ws) == 0
        t.device_status()
        ref = reference(want, q2, k, v, ids, 200)
        assert ((o[:rows].cpu().double() - ref[0]).abs() <= error_bound(ref, D, dtype)).all()


@pytest.mark.parametrize("field", ["num_seqs", "max_tokens", "max_blocks"])
@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (8, 2, 64, 16, "f32")], ids=str)
def test_tables_of_other_sizes(rbkv, shape, field):
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 200, *MIXED)
    tables = rbkv._StepTables.from_buffer_copy(t._tables)
    setattr(tables, field, getattr(tables, field) - 1)
    o = torch.full_like(q, 7.0, device="cuda")
    ws = torch.zeros(1 << 28, dtype=torch.uint8, device="cuda")
    assert _attention(rbkv, t, t.config, tables, q.cuda(), kd, vd, i32(ids), 200, o, ws) == 0
    _refused(rbkv, t)
    assert (o == 7.0).all()


@pytest.mark.parametrize("change", ["block", "rows"])
def test_append_of_another_shape(rbkv, change):
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, 8, 2, 64, 16, "f32", 0, *MIXED)
    tables = rbkv._StepTables.from_buffer_copy(t._tables)
    cfg = rbkv.Config(8, 2, 64, 16 if change == "rows" else 8, "f32", t.config.num_blocks)
    if change == "rows":
        tables.max_tokens -= 1
    new = torch.zeros(t.max_tokens, 2, 64, device="cuda")
    before = kd.clone(), vd.clone()
    assert rbkv.lib().rbkv_step_append(C.byref(cfg._c()), C.byref(tables), new.data_ptr(),
                                       new.data_ptr(), kd.data_ptr(), vd.data_ptr(), None) == 0
    _refused(rbkv, t)
    assert torch.equal(kd, before[0]) and torch.equal(vd, before[1])


@pytest.mark.parametrize("change", ["block", "pool", "num_seqs", "max_blocks"])
def test_release_of_another_shape(rbkv, change):
    t, want, *_ = _case(rbkv, 8, 2, 64, 16, "f32", 0, *MIXED)
    tables = rbkv._StepTables.from_buffer_copy(t._tables)
    blocks = t.config.num_blocks
    cfg = rbkv.Config(8, 2, 64, 8 if change == "block" else 16, "f32",
                      blocks - 1 if change == "pool" else blocks)
    if change in ("num_seqs", "max_blocks"):
        setattr(tables, change, getattr(tables, change) - 1)
    done = i32(np.ones(t.num_seqs))
    free, ctx = t.free.clone(), t.ctx.clone()
    assert rbkv.lib().rbkv_step_release(C.byref(cfg._c()), C.byref(tables), done.data_ptr(),
                                        None) == 0
    _refused(rbkv, t)
    assert torch.equal(t.free, free) and torch.equal(t.ctx, ctx)
    t.release(done)
    t.device_status()
    assert t.ctx.tolist() == [0] * t.num_seqs


def test_before_the_first_step(rbkv):
    """Tables that no step was built on: nothing to do, nothing to report."""
    cfg = rbkv.Config(8, 2, 128, 16, "bf16", 8)
    t = rbkv.StepTables(cfg, 3, 2, 5)
    kc = torch.zeros(cfg.cache_shape(), dtype=torch.bfloat16, device="cuda")
    q = torch.zeros(5, 8, 128, dtype=torch.bfloat16, device="cuda")
    kv = torch.ones(5, 2, 128, dtype=torch.bfloat16, device="cuda")
    o = torch.full_like(q, 7.0)
    t.append(kv, kv, kc, kc.clone())
    t.attention(q, kc, kc, prefix_table=i32([1]), prefix_len=9, o=o)
    t.device_status()
    assert (o == 7.0).all() and (kc == 0).all()
    t.block_table[1, 0] = 5                      # a request taken over from elsewhere
    t.free.fill_(0)
    t.ctx.copy_(i32([0, 10, 0]))
    t.release(i32([0, 1, 0]))
    t.device_status()
    assert t.free.tolist() == [1 << 5] and t.ctx.tolist() == [0, 0, 0]


def test_an_output_over_the_queries_is_refused(rbkv):
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, 8, 2, 64, 16, "f32", 20, [3, 0], [1, 40])
    both = torch.cat([q, q[:1]]).cuda()
    before = both.clone()
    for x, o in ((both[:-1], both[1:]), (both[1:], both[:-1])):
        with pytest.raises(rbkv.RbkvError) as e:
            t.attention(x, kd, vd, prefix_table=i32(ids), prefix_len=20, o=o)
        assert e.value.status == INVALID
    need = t.workspace_bytes(20)
    if need:
        with pytest.raises(rbkv.RbkvError):
            t.attention(both[:-1], kd, vd, prefix_table=i32(ids), prefix_len=20,
                        workspace=both.view(torch.uint8))
    torch.cuda.synchronize()
    assert torch.equal(both, before)


@pytest.mark.parametrize("shape", [(32, 8, 128, 64, "bf16"), (8, 2, 64, 16, "f32")], ids=str)
def test_a_workspace_is_needed_and_kept_apart(rbkv, shape):
    """One row behind a long prefix takes a workspace on every route: none, one
    that is too small and one that holds an operand are refused."""
    t, want, q, kd, vd, kc, vc, ids, rows = _case(rbkv, *shape, 3000, [300], [1])
    need, qc, idc = t.workspace_bytes(3000), q.cuda(), i32(ids)
    assert need > 0
    L, cfg = rbkv.lib(), t.config._c()
    ws, o = torch.zeros(need, dtype=torch.uint8, device="cuda"), torch.full_like(qc, 7.0)

    def call(ws, size, q=qc, o=o):
        return L.rbkv_step_attention(C.byref(cfg), C.byref(t._tables), q.data_ptr(),
                                     kd.data_ptr(), vd.data_ptr(), idc.data_ptr(), 3000,
                                     o.data_ptr(), ws, size, None)

    assert call(None, 0) == WORKSPACE and call(ws.data_ptr(), need - 1) == WORKSPACE
    inside = ws[need // 2 // 256 * 256:][:qc.nbytes].view(qc.dtype).view(qc.shape)
    assert call(ws.data_ptr(), need, q=inside) == INVALID
    assert call(ws.data_ptr(), need, o=inside) == INVALID
    torch.cuda.synchronize()
    assert (o == 7.0).all() and (ws == 0).all()
    assert call(ws.data_ptr(), need) == 0
    t.device_status()
    ref = reference(want, q, kc, vc, ids, 3000)
    assert ((o.cpu().double() - ref[0]).abs() <= error_bound(ref, shape[2], shape[4])).all()


def test_status_is_read_and_cleared_in_its_stream_order(rbkv):
    """A step that fails right behind a status read on a side stream: the words
    are cleared before its kernel, not after it."""
    t = rbkv.StepTables(rbkv.Config(8, 2, 64, 16, "f32", 8), 1, 4, 4)
    bad, good, one = i32([-1]), i32([0]), i32([1])
    side, busy = torch.cuda.Stream(), torch.zeros(1 << 26, device="cuda")
    torch.cuda.synchronize()
    for i in range(200):
        busy.add_(1.0)                           # the default stream has work of its own
        t.build(bad, one, stream=side)
        with pytest.raises(rbkv.RbkvError) as e:
            t.device_status(stream=side)
        assert e.value.status == INVALID, i
    t.build(good, one, stream=side)
    t.device_status(stream=side)


def test_workspace_bytes_of_refused_prefixes(rbkv):
    t = rbkv.StepTables(rbkv.Config(32, 8, 128, 64, "bf16", 8), 2, 4, 40)
    assert t.workspace_bytes(0) > 0 and t.workspace_bytes(1 << 30) > 0
    assert t.workspace_bytes(-1) == 0 and t.workspace_bytes((1 << 30) + 1) == 0
