"""The decoder layer's own steps without a GPU, over a library that only notes its calls."""
import pytest
import torch

from ragged_blocked_kv_gb300.layer import DecoderLayer


class _Noted:
    """Stands in for the library: every call is noted, nothing is computed."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *args, **kw: self.calls.append(name)


def _layer(rotary):
    lib = _Noted()
    weights = {n: torch.zeros(128, 128) for n in ("g_attn", "w_qkv", "w_o", "g_mlp", "w_gu", "w_down")}
    x = torch.zeros(3, 128)
    buf = {"a": x, "h": x, "b": x, "act": x, "gemm_ws": None,
           **{n: torch.zeros(3, 1, 128) for n in ("q", "k", "v", "o")}}
    return DecoderLayer(lib, weights, 1, 1, 128, rotary=rotary), lib, x, buf


def test_forward_into_hands_over_its_rotary_positions():
    rotary, seen = object(), []
    layer, lib, x, buf = _layer(rotary)
    layer.forward_into(x, x, buf, lambda q, k, v, o, rotary: seen.append(rotary), 3)
    assert seen == [rotary] and lib.calls == ["rmsnorm", "gemm_qkv", "gemm", "rmsnorm", "gemm", "gemm"]


def test_forward_into_refuses_a_callback_without_them():
    layer, lib, x, buf = _layer(object())
    with pytest.raises(TypeError, match="rotary"):
        layer.forward_into(x, x, buf, lambda q, k, v, o: None, 3)
    assert lib.calls == ["rmsnorm", "gemm_qkv"]


def test_forward_into_without_rotary_positions():
    seen = []
    layer, lib, x, buf = _layer(None)
    layer.forward_into(x, x, buf, lambda q, k, v, o: seen.append(q.shape), 3)
    assert seen == [(3, 1, 128)]
