"""The decoder layer with rotary positions in its fixed-buffer form."""
import numpy as np
import pytest
import torch

from test_gpu_rotary import _close

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
def test_forward_into_rotates(rbkv, captured):
    """forward_into hands its rotary positions to the callback, over a pass and over a frame
    in a captured graph."""
    from ragged_blocked_kv_gb300.layer import DecoderLayer, random_weights
    hidden, hq, hkv, D, ffn, T = 512, 4, 2, 128, 512, 205
    w = random_weights(hidden, hq, hkv, D, ffn, seed=1)
    cfg = rbkv.Config(hq, hkv, D, 64, "bf16", 16)
    rope = rbkv.Rotary(D)
    x = torch.randn(T, hidden, generator=torch.Generator().manual_seed(3)).bfloat16().cuda()
    kc, vc, kp, vp = (torch.zeros(cfg.cache_shape(), dtype=torch.bfloat16, device="cuda")
                      for _ in range(4))
    p = rbkv.Composer(cfg).compose(300, 0, [(1, 200, 0), (2, 5, 0)])
    frame = rbkv.Frame(cfg, T, packed_units=1)
    p.set_chunk_items(frame.chunk_items)
    ws = torch.empty(max(256, frame.workspace_bytes()), dtype=torch.uint8, device="cuda")

    def plain(q, k, v, o):
        rbkv.kv_append(p, k, v, kp, vp)
        rbkv.ragged_attention(p, q, kp, vp, o=o)

    def over_pass(q, k, v, o, rotary):
        assert rotary is rope
        rbkv.kv_append_rotary(p, rotary, q, k, v, kc, vc, q_out=q)
        rbkv.ragged_attention(p, q, kc, vc, o=o)

    def over_frame(q, k, v, o, rotary):
        assert rotary is rope
        frame.kv_append_rotary(rotary, q, k, v, kc, vc, q_out=q)
        frame.attention(q, kc, vc, o, ws)

    before, raw = torch.empty_like(x), DecoderLayer(rbkv, w, hq, hkv, D)
    raw_buf = raw.buffers(T)
    raw.forward_into(x, before, raw_buf, plain, T)       # (no rotary positions: as ever)
    layer = DecoderLayer(rbkv, w, hq, hkv, D, rotary=rope)
    out, buf = torch.empty_like(x), layer.buffers(T)
    if captured:
        frame.load(p)
        layer.forward_into(x, out, buf, over_frame, T)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            layer.forward_into(x, out, buf, over_frame, T)
        for y in (out, kc, vc):
            y.zero_()
        graph.replay()
        frame.device_status()
    else:
        layer.forward_into(x, out, buf, over_pass, T)
    p.device_status()
    position = np.concatenate([np.arange(200), np.arange(5)])
    slot = torch.from_numpy(p.meta.slot.astype(np.int64))
    _close(buf["q"], raw_buf["q"].cpu(), position, rope, "bf16")
    _close(kc.cpu()[slot // 64, :, slot % 64], raw_buf["k"].cpu(), position, rope, "bf16")
    assert torch.equal(vc, vp)
    assert torch.equal(buf["o"], rbkv.ragged_attention(p, buf["q"], kc, vc))
    first = [0, 200]                                     # one key: position changes nothing
    assert torch.equal(out[first], before[first]) and not torch.equal(out[100], before[100])


def test_a_callback_without_rotary_positions_is_refused(rbkv):
    """A callback that takes none would give a layer with rotary positions rows that were
    not turned: it fails, and nothing is written behind it."""
    from ragged_blocked_kv_gb300.layer import DecoderLayer, random_weights
    w = random_weights(256, 2, 1, 128, 256, seed=1)
    layer = DecoderLayer(rbkv, w, 2, 1, 128, rotary=rbkv.Rotary(128))
    x = torch.randn(4, 256).bfloat16().cuda()
    out = torch.full_like(x, 7.0)
    with pytest.raises(TypeError, match="rotary"):
        layer.forward_into(x, out, layer.buffers(4), lambda q, k, v, o: o.zero_(), 4)
    assert (out == 7.0).all()
