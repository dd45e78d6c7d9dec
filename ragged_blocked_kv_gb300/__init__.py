"""Python binding of librbkv (ctypes; argument marshalling only).

Every step of the pass runs in the library: composition, block allocation and
split planning in its host C++ code, appending and attention in its sm_103a
kernels.  This module turns torch tensors into device pointers and streams into
handles, and raises on a non-OK status.  There is no fallback: if the library
is missing, importing the names below raises.

    cfg = Config(num_heads_q=32, num_heads_kv=8, head_dim=128, block_size=64,
                 dtype="bf16", num_blocks=4096)
    comp = Composer(cfg)
    p = comp.compose(budget=2048, max_chunk=768, states=[(seq_id, prompt_len, seen), ...])
    kv_append(p, k_new, v_new, k_cache, v_cache)
    o = ragged_attention(p, q, k_cache, v_cache)
"""
from __future__ import annotations

import ctypes as C
import math
from dataclasses import dataclass
from pathlib import Path
from typing import List, Optional, Sequence, Tuple

import numpy as np

_LIB_PATH = Path(__file__).resolve().parent / "_lib" / "librbkv.so"

OK, ERR_INVALID, ERR_NO_BLOCKS, ERR_CUDA, ERR_DEVICE_BOUNDS, ERR_UNSUPPORTED, ERR_WORKSPACE, \
    ERR_TIMEOUT = 0, -1, -2, -3, -4, -5, -6, -7
BF16, F32 = 0, 1


class RbkvError(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(f"rbkv status {status}: {message}")
        self.status = status


class NoBlocksError(RbkvError):
    pass


class _Config(C.Structure):
    _fields_ = [("num_heads_q", C.c_int32), ("num_heads_kv", C.c_int32), ("head_dim", C.c_int32),
                ("block_size", C.c_int32), ("dtype", C.c_int32), ("num_blocks", C.c_int32)]


class _SeqState(C.Structure):
    _fields_ = [("seq_id", C.c_int64), ("prompt_len", C.c_int32), ("seen", C.c_int32)]


class _PassMeta(C.Structure):
    _fields_ = [("num_seqs", C.c_int32), ("num_tokens", C.c_int32), ("num_block_ids", C.c_int32),
                ("block_size", C.c_int32),
                ("seq_ids", C.POINTER(C.c_int64)), ("q_start", C.POINTER(C.c_int32)),
                ("n_new", C.POINTER(C.c_int32)), ("seen", C.POINTER(C.c_int32)),
                ("ctx", C.POINTER(C.c_int32)), ("block_start", C.POINTER(C.c_int32)),
                ("block_ids", C.POINTER(C.c_int32)), ("slot", C.POINTER(C.c_int32))]


class _PlanInfo(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "num_sms", "decode_rows", "decode_items", "max_splits", "split_keys", "partials",
        "chunk_rows", "chunk_tiles", "generic_items", "fast_decode", "fast_chunk",
        "chunk_items", "chunk_single", "chunk_steps_total", "chunk_steps_max",
        "decode_grid", "decode_keys_total", "decode_keys_max")]


class _FrameCaps(C.Structure):
    _fields_ = [(n, C.c_int32) for n in (
        "max_tokens", "max_seqs", "max_blocks", "max_decode_items", "max_chunk_tiles",
        "max_combine_rows", "max_parts", "packed_units", "chunk_items")]


class _StepTables(C.Structure):
    _fields_ = [("num_seqs", C.c_int32), ("max_blocks", C.c_int32), ("max_tokens", C.c_int32)] + \
        [(n, C.c_void_p) for n in ("block_table", "free_words", "q_start", "ctx", "position",
                                   "slot", "plan", "status")]


class _StepDraft(C.Structure):
    _fields_ = [(n, C.c_void_p) for n in ("place", "ancestors", "path", "accepted", "next_token",
                                          "work")]


class _Rotary(C.Structure):
    _fields_ = [("turns", C.c_void_p), ("rotary_dim", C.c_int32), ("interleaved", C.c_int32),
                ("scale", C.c_float)]


# Every symbol include/rbkv.h declares, with (restype, argtypes).
_P = C.c_void_p
SIGNATURES = {
    "rbkv_abi_version": (C.c_int32, []),
    "rbkv_last_error": (C.c_char_p, []),
    "rbkv_composer_create": (C.c_int, [C.POINTER(_Config), C.POINTER(_P)]),
    "rbkv_composer_destroy": (None, [_P]),
    "rbkv_compose_pass": (C.c_int, [_P, C.c_int32, C.c_int32, C.POINTER(_SeqState), C.c_int32,
                                    C.POINTER(_P)]),
    "rbkv_release_seq": (C.c_int, [_P, C.c_int64]),
    "rbkv_compose_pass_policy": (C.c_int, [_P, C.c_int32, C.c_int32, C.c_int32,
                                           C.POINTER(_SeqState), C.c_int32, C.POINTER(_P)]),
    "rbkv_budget_for_latency": (C.c_int32, [C.POINTER(C.c_int32), C.POINTER(C.c_double),
                                            C.c_int32, C.c_double]),
    "rbkv_latency_at": (C.c_double, [C.POINTER(C.c_int32), C.POINTER(C.c_double), C.c_int32,
                                     C.c_int32]),
    "rbkv_pass_rollback": (C.c_int, [_P, _P]),
    "rbkv_composer_free_blocks": (C.c_int32, [_P]),
    "rbkv_pass_get_meta": (C.c_int, [_P, C.POINTER(_PassMeta)]),
    "rbkv_pass_set_split_keys": (C.c_int, [_P, C.c_int32]),
    "rbkv_pass_set_chunk_items": (C.c_int, [_P, C.c_int32]),
    "rbkv_pass_get_plan": (C.c_int, [_P, C.POINTER(_PlanInfo)]),
    "rbkv_pass_plan_for_sms": (C.c_int, [_P, C.c_int32, C.POINTER(_PlanInfo)]),
    "rbkv_pass_destroy": (None, [_P]),
    "rbkv_kv_append": (C.c_int, [_P, _P, _P, _P, _P, _P]),
    "rbkv_kv_append_rotary": (C.c_int, [_P, C.POINTER(_Rotary), _P, _P, _P, _P, _P, _P, _P]),
    "rbkv_attention_workspace_bytes": (C.c_size_t, [_P]),
    "rbkv_ragged_attention": (C.c_int, [_P, _P, _P, _P, _P, _P, C.c_size_t, _P]),
    "rbkv_pass_device_status": (C.c_int, [_P, _P]),
    "rbkv_ragged_attention_noalloc": (C.c_int, [_P, _P, _P, _P, _P, _P]),
    "rbkv_frame_create": (C.c_int, [C.POINTER(_Config), C.POINTER(_FrameCaps), C.POINTER(_P),
                                    C.POINTER(_FrameCaps)]),
    "rbkv_frame_destroy": (None, [_P]),
    "rbkv_frame_load": (C.c_int, [_P, _P, _P]),
    "rbkv_frame_kv_append": (C.c_int, [_P, _P, _P, _P, _P, _P]),
    "rbkv_frame_kv_append_rotary": (C.c_int, [_P, C.POINTER(_Rotary), _P, _P, _P, _P, _P, _P,
                                              _P]),
    "rbkv_frame_workspace_bytes": (C.c_size_t, [_P]),
    "rbkv_frame_attention": (C.c_int, [_P, _P, _P, _P, _P, _P, C.c_size_t, _P]),
    "rbkv_frame_device_status": (C.c_int, [_P, _P]),
    "rbkv_debug_corrupt_pass": (C.c_int, [_P, C.c_int32, C.c_int32, C.c_int32]),
    "rbkv_debug_wait_timeout": (C.c_int, [_P, C.c_int64, _P]),
    "rbkv_kernel_launches": (C.c_int64, []),
    "rbkv_profile_enable": (None, [C.c_int32]),
    "rbkv_profile_read": (C.c_int, [C.c_int32, C.POINTER(C.c_double), C.POINTER(C.c_int64)]),
    "rbkv_profile_reset": (None, []),
    "rbkv_gemm_bf16": (C.c_int, [_P, _P, _P, C.c_int64, C.c_int64, C.c_int64, _P, C.c_int32,
                                 _P, C.c_size_t, _P, _P]),
    "rbkv_gemm_workspace_bytes": (C.c_size_t, [C.c_int64, C.c_int64, C.c_int64]),
    "rbkv_rmsnorm_bf16": (C.c_int, [_P, _P, _P, C.c_int64, C.c_int64, C.c_float, _P]),
    "rbkv_gemm_bf16_qkv": (C.c_int, [_P, _P, _P, _P, _P, C.c_int64, C.c_int64, C.c_int64,
                                     C.c_int64, _P, C.c_size_t, _P, _P]),
    "rbkv_step_plan_ints": (C.c_int64, [C.c_int32, C.c_int32]),
    "rbkv_step_build": (C.c_int, [C.POINTER(_Config), C.POINTER(_StepTables), _P, _P, _P, _P,
                                  _P]),
    "rbkv_step_release": (C.c_int, [C.POINTER(_Config), C.POINTER(_StepTables), _P, _P]),
    "rbkv_step_append": (C.c_int, [C.POINTER(_Config), C.POINTER(_StepTables), _P, _P, _P, _P,
                                   _P]),
    "rbkv_step_workspace_bytes": (C.c_size_t, [C.POINTER(_Config), C.POINTER(_StepTables),
                                               C.c_int32]),
    "rbkv_step_attention": (C.c_int, [C.POINTER(_Config), C.POINTER(_StepTables), _P, _P, _P, _P,
                                      C.c_int32, _P, _P, C.c_size_t, _P]),
    "rbkv_step_draft_plan": (C.c_int, [C.POINTER(_Config), C.POINTER(_StepTables),
                                       C.POINTER(_StepDraft), _P, _P]),
    "rbkv_step_append_rotary": (C.c_int, [C.POINTER(_Config), C.POINTER(_StepTables),
                                          C.POINTER(_StepDraft), C.POINTER(_Rotary), C.c_int32,
                                          _P, _P, _P, _P, _P, _P, _P]),
    "rbkv_step_attention_draft": (C.c_int, [C.POINTER(_Config), C.POINTER(_StepTables),
                                            C.POINTER(_StepDraft), _P, _P, _P, _P, C.c_int32, _P,
                                            _P, C.c_size_t, _P]),
    "rbkv_step_draft_accept": (C.c_int, [C.POINTER(_Config), C.POINTER(_StepTables),
                                         C.POINTER(_StepDraft), _P, _P, _P, _P]),
    "rbkv_step_draft_compact": (C.c_int, [C.POINTER(_Config), C.POINTER(_StepTables),
                                          C.POINTER(_StepDraft), _P, _P, _P]),
    "rbkv_step_device_status": (C.c_int, [C.POINTER(_StepTables), _P]),
    "rbkv_router_create": (C.c_int, [C.c_int32, C.POINTER(_P)]),
    "rbkv_router_destroy": (None, [_P]),
    "rbkv_router_assign": (C.c_int, [_P, C.c_int64, C.c_int32, C.c_int32,
                                     C.POINTER(C.c_int32)]),
    "rbkv_router_progress": (C.c_int, [_P, C.c_int64, C.c_int32]),
    "rbkv_router_finish": (C.c_int, [_P, C.c_int64]),
    "rbkv_router_load": (C.c_int64, [_P, C.c_int32]),
    "rbkv_router_active": (C.c_int32, [_P, C.c_int32]),
}

KERNEL_KINDS = {"kv_append": 0, "chunk": 1, "decode": 2, "generic": 3, "combine": 4,
                "upload": 5}

_lib = None


def library_path() -> Path:
    return _LIB_PATH


def lib():
    """The loaded librbkv (raises if it was not built)."""
    global _lib
    if _lib is None:
        if not _LIB_PATH.exists():
            raise ImportError(
                f"{_LIB_PATH} is missing; build it with `python -m ragged_blocked_kv_gb300.build` "
                "(there is no fallback implementation)")
        L = C.CDLL(str(_LIB_PATH))
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def _check(status: int):
    if status != OK:
        msg = lib().rbkv_last_error().decode(errors="replace")
        if status == ERR_NO_BLOCKS:
            raise NoBlocksError(status, msg)
        raise RbkvError(status, msg)


@dataclass(frozen=True)
class Config:
    num_heads_q: int
    num_heads_kv: int
    head_dim: int
    block_size: int
    dtype: str          # "bf16" or "f32"
    num_blocks: int

    def _c(self) -> _Config:
        return _Config(self.num_heads_q, self.num_heads_kv, self.head_dim, self.block_size,
                       BF16 if self.dtype == "bf16" else F32, self.num_blocks)

    @property
    def torch_dtype(self):
        import torch
        return torch.bfloat16 if self.dtype == "bf16" else torch.float32

    def cache_shape(self) -> Tuple[int, int, int, int]:
        return (self.num_blocks, self.num_heads_kv, self.block_size, self.head_dim)


@dataclass
class PassMeta:
    seq_ids: np.ndarray
    q_start: np.ndarray
    n_new: np.ndarray
    seen: np.ndarray
    ctx: np.ndarray
    block_start: np.ndarray
    block_ids: np.ndarray
    slot: np.ndarray

    @property
    def num_tokens(self) -> int:
        return int(self.q_start[-1])

    @property
    def num_seqs(self) -> int:
        return len(self.seq_ids)


def _arr(ptr, n, dtype):
    if n == 0:
        return np.zeros(0, dtype)
    return np.ctypeslib.as_array(ptr, shape=(n,)).astype(dtype, copy=True)


class Pass:
    """One composed pass (owns its library handle)."""

    def __init__(self, handle: int, config: Config):
        self._h = _P(handle)
        self.config = config
        self._view = _PassMeta()
        _check(lib().rbkv_pass_get_meta(self._h, C.byref(self._view)))
        self.num_tokens = int(self._view.num_tokens)
        self._meta = None

    @property
    def meta(self) -> PassMeta:
        """Copies of the pass's metadata arrays (made on first access)."""
        if self._meta is None:
            m = self._view
            S, T = m.num_seqs, m.num_tokens
            self._meta = PassMeta(_arr(m.seq_ids, S, np.int64), _arr(m.q_start, S + 1, np.int32),
                                  _arr(m.n_new, S, np.int32), _arr(m.seen, S, np.int32),
                                  _arr(m.ctx, S, np.int32), _arr(m.block_start, S + 1, np.int32),
                                  _arr(m.block_ids, m.num_block_ids, np.int32),
                                  _arr(m.slot, T, np.int32))
        return self._meta

    def set_split_keys(self, keys: int) -> None:
        _check(lib().rbkv_pass_set_split_keys(self._h, int(keys)))

    def set_chunk_items(self, mode: str) -> None:
        """Group prompt-chunk tiles as "auto", "pairs" or "single" work items."""
        m = {"auto": 0, "pairs": 1, "single": 2}[mode]
        _check(lib().rbkv_pass_set_chunk_items(self._h, m))

    def plan(self) -> dict:
        info = _PlanInfo()
        _check(lib().rbkv_pass_get_plan(self._h, C.byref(info)))
        return {n: getattr(info, n) for n, _ in _PlanInfo._fields_}

    def plan_for_sms(self, num_sms: int) -> dict:
        info = _PlanInfo()
        _check(lib().rbkv_pass_plan_for_sms(self._h, int(num_sms), C.byref(info)))
        return {n: getattr(info, n) for n, _ in _PlanInfo._fields_}

    def workspace_bytes(self) -> int:
        return int(lib().rbkv_attention_workspace_bytes(self._h))

    def device_status(self, stream=None) -> None:
        _check(lib().rbkv_pass_device_status(self._h, _stream(stream)))

    def debug_corrupt(self, which: str, index: int, value: int) -> None:
        """Fault injection for tests: overwrite a block-table ("block") or
        slot ("slot") entry before the pass reaches the device."""
        w = {"block": 0, "slot": 1}[which]
        _check(lib().rbkv_debug_corrupt_pass(self._h, w, int(index), int(value)))

    def debug_wait_timeout(self, limit_cycles: int, stream=None) -> None:
        """Run a bounded wait that is bound to give up (reported in the status)."""
        _check(lib().rbkv_debug_wait_timeout(self._h, int(limit_cycles), _stream(stream)))

    def destroy(self) -> None:
        if self._h:
            lib().rbkv_pass_destroy(self._h)
            self._h = _P(None)

    def __del__(self):
        try:
            self.destroy()
        except Exception:
            pass


class SeqStates:
    """A request list in the library's layout (see ``seq_states``)."""

    def __init__(self, arr, n):
        self.arr, self.n = arr, n


def seq_states(states: Sequence[Tuple[int, int, int]]) -> SeqStates:
    arr = (_SeqState * max(1, len(states)))()
    for i, (sid, plen, seen) in enumerate(states):
        arr[i] = _SeqState(int(sid), int(plen), int(seen))
    return SeqStates(arr, len(states))


class Composer:
    """Dynamic SplitFuse composer and block pool of one cache layout."""

    def __init__(self, config: Config):
        self.config = config
        h = _P()
        cfg = config._c()
        _check(lib().rbkv_composer_create(C.byref(cfg), C.byref(h)))
        self._h = h

    def compose(self, budget: int, max_chunk: int, states, policy: str = "greedy") -> Pass:
        """``states``: [(seq_id, prompt_len, seen), ...] in list order, or an
        array made once with ``seq_states`` (cheaper when reused).  ``policy``:
        "greedy" (fill the budget) or "equal" (near-equal prompt chunks)."""
        if not isinstance(states, SeqStates):
            states = seq_states(states)
        out = _P()
        if policy == "greedy":
            _check(lib().rbkv_compose_pass(self._h, int(budget), int(max_chunk), states.arr,
                                           states.n, C.byref(out)))
        else:
            pol = {"equal": 1}.get(policy, -1)
            _check(lib().rbkv_compose_pass_policy(self._h, int(budget), int(max_chunk), pol,
                                                  states.arr, states.n, C.byref(out)))
        return Pass(out.value, self.config)

    def rollback(self, p: Pass) -> None:
        """Undo what composing ``p`` did to the pool and the recorded contexts
        (newest pass first)."""
        _check(lib().rbkv_pass_rollback(self._h, p._h))

    def release(self, seq_id: int) -> None:
        _check(lib().rbkv_release_seq(self._h, int(seq_id)))

    def free_blocks(self) -> int:
        return int(lib().rbkv_composer_free_blocks(self._h))

    def close(self) -> None:
        if self._h:
            lib().rbkv_composer_destroy(self._h)
            self._h = _P(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


def _stream(stream):
    if isinstance(stream, _P):
        return stream
    if stream is None:
        import torch
        return _P(torch.cuda.current_stream().cuda_stream)
    if isinstance(stream, int):
        return _P(stream)
    return _P(stream.cuda_stream)


def _device_calls():
    """(index of the current device, handle of a device's current stream): the
    short ways where torch has them."""
    import torch
    current = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
    stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                     lambda index: torch.cuda.current_stream(index).cuda_stream)
    return current, stream


def _device(device):
    import torch
    return torch.cuda.device(device)


def _int32(x: int, name: str) -> int:
    """(ctypes would cut it off)"""
    if not -2 ** 31 <= x < 2 ** 31:
        raise ValueError(f"{name} must fit in 32 bits")
    return x


def _dev_ptr(t, name, dtype, shape):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return _P(t.data_ptr())


def kv_append(p: Pass, k_new, v_new, k_cache, v_cache, stream=None) -> None:
    """Scatter the pass's new K/V rows into the blocked caches (in place)."""
    c = p.config
    T = p.num_tokens
    dt = c.torch_dtype
    row = (T, c.num_heads_kv, c.head_dim)
    _check(lib().rbkv_kv_append(p._h, _dev_ptr(k_new, "k_new", dt, row),
                                _dev_ptr(v_new, "v_new", dt, row),
                                _dev_ptr(k_cache, "k_cache", dt, c.cache_shape()),
                                _dev_ptr(v_cache, "v_cache", dt, c.cache_shape()),
                                _stream(stream)))


class _Arrays:
    """An object whose device arrays the library holds by address."""

    _HELD = frozenset()
    _HOW = "write into it (copy_, fill_, ...)"

    def __setattr__(self, name, value):
        # (plain attributes, for fast reads: a small step's time is the host's)
        if name in self._HELD and self.__dict__.get(name, value) is not value:
            raise AttributeError(f"{name} cannot be replaced: {self._HOW}")
        object.__setattr__(self, name, value)

    def __delattr__(self, name):
        if name in self._HELD:
            raise AttributeError(f"{name} cannot be deleted")
        object.__delattr__(self, name)


class Rotary(_Arrays):
    """A rotary position embedding: the table of its angles per position, on the GPU.

    Pair i of a head's first ``rotary_dim`` elements (i and i + rotary_dim / 2 for
    ``layout="half"``, 2 i and 2 i + 1 for ``"interleaved"``) turns by position *
    theta_i, theta_i = base ** (-2 i / rotary_dim), and is multiplied by ``scale``;
    the other elements stay.  ``scaling`` stretches contexts by ``factor``:
    "linear" divides every theta_i; "base" raises the base to base * factor **
    (rotary_dim / (rotary_dim - 2)); "parts" divides those pairs that turn less than
    ``low`` times over ``original_length`` positions, leaves those that turn more than
    ``high`` times, and blends in between.  ``inv_freq``: the theta_i themselves
    (fp64 values) instead.

        rope = Rotary(128, base=500000.0)
        q = t.append_rotary(rope, q, k_new, v_new, k_cache, v_cache)

    Angles are kept as 64-bit fractions of a turn: far positions lose nothing.  The
    table is written by the stream that is current here, in the constructor.  Calls hold
    its address and the other values as they were then: for others make another Rotary.
    """

    LAYOUTS = {"half": 0, "interleaved": 1}
    _HELD = frozenset(("rotary_dim", "layout", "scale", "inv_freq", "turns"))
    _HOW = "make another Rotary"

    def __init__(self, rotary_dim: int, base: float = 10000.0, layout: str = "half",
                 scaling: str = "none", factor: float = 1.0, original_length: int = 0,
                 low: float = 1.0, high: float = 32.0, scale: float = 1.0, inv_freq=None,
                 device="cuda"):
        import torch
        self.rotary_dim, self.layout, self.scale = int(rotary_dim), layout, float(scale)
        if self.rotary_dim < 2 or self.rotary_dim % 2 or self.rotary_dim > 256:
            raise ValueError("rotary_dim must be even, in [2, 256]")
        if layout not in self.LAYOUTS:
            raise ValueError("layout must be 'half' or 'interleaved'")
        if not math.isfinite(C.c_float(self.scale).value):
            raise ValueError("scale must be finite in fp32")
        if inv_freq is not None:
            theta = np.array(inv_freq, np.float64)
            if theta.shape != (self.rotary_dim // 2,) or not np.isfinite(theta).all():
                raise ValueError("inv_freq must be rotary_dim / 2 finite values")
            if scaling != "none":
                raise ValueError("inv_freq takes no scaling")
        else:
            try:
                theta = self._theta(float(base), scaling, float(factor), original_length, low,
                                    high)
            except OverflowError:
                raise ValueError("angles per position are out of range") from None
        if not (np.abs(theta) < 2.0 ** 900).all():
            raise ValueError("angles per position are out of range")
        theta.setflags(write=False)
        self.inv_freq = theta
        turns = [round(math.ldexp(float(x) / (2 * math.pi), 64)) % 2 ** 64 for x in theta]
        self.turns = torch.tensor([x - 2 ** 64 if x >= 2 ** 63 else x for x in turns],
                                  dtype=torch.int64, device=device)
        self._bind()

    def _bind(self):
        self._c = C.byref(_Rotary(self.turns.data_ptr(), self.rotary_dim,
                                  self.LAYOUTS[self.layout], self.scale))
        self._device = self.turns.device

    # (copies hold the address of their own table)
    def __getstate__(self):
        return {name: self.__dict__[name] for name in self._HELD}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self.inv_freq.setflags(write=False)
        self._bind()

    def _theta(self, base, scaling, factor, original_length, low, high):
        R = self.rotary_dim
        if not (base > 0 and factor > 0 and math.isfinite(base) and math.isfinite(factor)):
            raise ValueError("base and factor must be positive")
        if scaling == "base":
            base = base * factor ** (R / max(R - 2, 1))
        theta = base ** (-np.arange(0, R, 2, dtype=np.float64) / R)
        if scaling == "linear":
            theta = theta / factor
        elif scaling == "parts":
            if original_length < 1 or not high > low:
                raise ValueError("'parts' needs original_length >= 1 and high > low")
            turned = original_length * theta / (2 * math.pi)
            keep = np.clip((turned - low) / (high - low), 0.0, 1.0)
            theta = theta * (keep + (1.0 - keep) / factor)
        elif scaling not in ("none", "base"):
            raise ValueError("scaling must be 'none', 'linear', 'base' or 'parts'")
        return theta

    def _on(self, device):
        if self._device != device:
            raise ValueError(f"rotary is on {self._device}, the call on {device}")
        return self._c


def _empty_on(stream, shape, dtype, device):
    """An uninitialised tensor, allocated on the stream that uses it."""
    import torch
    with torch.cuda.device(device), \
            torch.cuda.stream(torch.cuda.ExternalStream(_stream(stream).value or 0, device)):
        return torch.empty(shape, dtype=dtype, device=device)


def _on_current(*tensors):
    """Tensors of a call that runs on the current device."""
    import torch
    for t in tensors:
        if t.get_device() != torch.cuda.current_device():
            raise ValueError(f"a tensor is on {t.device}, the call on the current device")


def kv_append_rotary(p: Pass, rotary: Rotary, q, k_new, v_new, k_cache, v_cache, q_out=None,
                     stream=None):
    """``kv_append`` with the rotation on the way: rotated keys and the values into the
    caches, rotated queries into ``q_out`` (which may be ``q``), by the rows' positions
    in their sequences; returns ``q_out`` ``[T][H_q][D]``."""
    c = p.config
    T, dt = p.num_tokens, c.torch_dtype
    row, qshape = (T, c.num_heads_kv, c.head_dim), (T, c.num_heads_q, c.head_dim)
    _on_current(q, k_new, v_new, k_cache, v_cache, *(() if q_out is None else (q_out,)))
    if q_out is None:
        q_out = _empty_on(stream, qshape, dt, q.device)
    _check(lib().rbkv_kv_append_rotary(p._h, rotary._on(q.device), _dev_ptr(q, "q", dt, qshape),
                                       _dev_ptr(q_out, "q_out", dt, qshape),
                                       _dev_ptr(k_new, "k_new", dt, row),
                                       _dev_ptr(v_new, "v_new", dt, row),
                                       _dev_ptr(k_cache, "k_cache", dt, c.cache_shape()),
                                       _dev_ptr(v_cache, "v_cache", dt, c.cache_shape()),
                                       _stream(stream)))
    return q_out


def ragged_attention(p: Pass, q, k_cache, v_cache, o=None, workspace=None, stream=None):
    """Ragged causal attention of every pass row; returns O ``[T][H_q][D]``."""
    import torch
    c = p.config
    T = p.num_tokens
    dt = c.torch_dtype
    qshape = (T, c.num_heads_q, c.head_dim)
    if o is None:
        o = torch.empty(qshape, dtype=dt, device=q.device)
    need = p.workspace_bytes()
    if need and workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=q.device)
    ws_ptr = _P(workspace.data_ptr()) if workspace is not None else _P(None)
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check(lib().rbkv_ragged_attention(p._h, _dev_ptr(q, "q", dt, qshape),
                                       _dev_ptr(k_cache, "k_cache", dt, c.cache_shape()),
                                       _dev_ptr(v_cache, "v_cache", dt, c.cache_shape()),
                                       _dev_ptr(o, "o", dt, qshape), ws_ptr, ws_bytes,
                                       _stream(stream)))
    return o


def ragged_attention_noalloc(p: Pass, q, k_cache, v_cache, o, stream=None):
    """Ragged attention with the library's own static scratch instead of a
    workspace: for callers that must not allocate device memory.  ``o`` must
    be given (this call allocates nothing) and the pass must already have been
    through ``kv_append``.  Calls that overlap on the GPU share the scratch and
    race; keep them ordered on one stream."""
    c = p.config
    T = p.num_tokens
    dt = c.torch_dtype
    qshape = (T, c.num_heads_q, c.head_dim)
    _check(lib().rbkv_ragged_attention_noalloc(p._h, _dev_ptr(q, "q", dt, qshape),
                                               _dev_ptr(k_cache, "k_cache", dt, c.cache_shape()),
                                               _dev_ptr(v_cache, "v_cache", dt, c.cache_shape()),
                                               _dev_ptr(o, "o", dt, qshape), _stream(stream)))
    return o


class Frame:
    """Fixed device home for one pass at a time, so that the append and
    attention launches are identical for every pass (capturable once as a CUDA
    graph and replayed).  ``load(pass)`` before each replay, on the same
    stream.  Q/K/V/O buffers have ``max_tokens`` rows; rows past the loaded
    pass's tokens are ignored."""

    CHUNK_ITEMS = {"auto": 0, "pairs": 1, "single": 2}

    def __init__(self, config: Config, max_tokens: int, **caps):
        if isinstance(caps.get("chunk_items"), str):
            caps["chunk_items"] = self.CHUNK_ITEMS[caps["chunk_items"]]
        want = _FrameCaps(max_tokens=int(max_tokens), **{k: int(v) for k, v in caps.items()})
        got = _FrameCaps()
        h = _P()
        _check(lib().rbkv_frame_create(C.byref(config._c()), C.byref(want), C.byref(h),
                                       C.byref(got)))
        self._h = h
        self.config = config
        self.caps = {n: getattr(got, n) for n, _ in _FrameCaps._fields_}
        self.max_tokens = self.caps["max_tokens"]
        # the grouping of chunk tiles every pass loaded here is planned with
        self.chunk_items = {1: "pairs", 2: "single"}[self.caps["chunk_items"]]

    def workspace_bytes(self) -> int:
        return int(lib().rbkv_frame_workspace_bytes(self._h))

    def load(self, p: "Pass", stream=None) -> None:
        _check(lib().rbkv_frame_load(self._h, p._h, _stream(stream)))

    def kv_append(self, k_new, v_new, k_cache, v_cache, stream=None) -> None:
        c = self.config
        dt = c.torch_dtype
        row = (self.max_tokens, c.num_heads_kv, c.head_dim)
        _check(lib().rbkv_frame_kv_append(self._h, _dev_ptr(k_new, "k_new", dt, row),
                                          _dev_ptr(v_new, "v_new", dt, row),
                                          _dev_ptr(k_cache, "k_cache", dt, c.cache_shape()),
                                          _dev_ptr(v_cache, "v_cache", dt, c.cache_shape()),
                                          _stream(stream)))

    def kv_append_rotary(self, rotary: Rotary, q, k_new, v_new, k_cache, v_cache, q_out=None,
                         stream=None):
        """``kv_append_rotary`` of the loaded pass; returns ``q_out`` ([max_tokens][H_q][D];
        rows past the pass's are left as they were)."""
        c = self.config
        dt = c.torch_dtype
        row = (self.max_tokens, c.num_heads_kv, c.head_dim)
        qshape = (self.max_tokens, c.num_heads_q, c.head_dim)
        _on_current(q, k_new, v_new, k_cache, v_cache, *(() if q_out is None else (q_out,)))
        if q_out is None:
            q_out = _empty_on(stream, qshape, dt, q.device)
        _check(lib().rbkv_frame_kv_append_rotary(
            self._h, rotary._on(q.device), _dev_ptr(q, "q", dt, qshape),
            _dev_ptr(q_out, "q_out", dt, qshape), _dev_ptr(k_new, "k_new", dt, row),
            _dev_ptr(v_new, "v_new", dt, row), _dev_ptr(k_cache, "k_cache", dt, c.cache_shape()),
            _dev_ptr(v_cache, "v_cache", dt, c.cache_shape()), _stream(stream)))
        return q_out

    def attention(self, q, k_cache, v_cache, o, workspace, stream=None) -> None:
        c = self.config
        dt = c.torch_dtype
        qshape = (self.max_tokens, c.num_heads_q, c.head_dim)
        _check(lib().rbkv_frame_attention(
            self._h, _dev_ptr(q, "q", dt, qshape),
            _dev_ptr(k_cache, "k_cache", dt, c.cache_shape()),
            _dev_ptr(v_cache, "v_cache", dt, c.cache_shape()), _dev_ptr(o, "o", dt, qshape),
            _P(workspace.data_ptr()), workspace.numel() * workspace.element_size(),
            _stream(stream)))

    def device_status(self, stream=None) -> None:
        _check(lib().rbkv_frame_device_status(self._h, _stream(stream)))

    def close(self) -> None:
        if getattr(self, "_h", None):
            lib().rbkv_frame_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


class StepTables(_Arrays):
    """Block tables, slots and the attention plan of a step, on the GPU.

    ``build`` makes them from device-side lengths, with no host work and no
    synchronisation, so that a decoding loop can be captured once as a CUDA
    graph and replayed; ``append`` and ``attention`` then run any number of
    layers on them.  The batch may share one prefix with a block list of its
    own (``prefix_table``), whose keys all rows attend together::

        t = StepTables(cfg, num_seqs, max_blocks, max_tokens)
        t.build(t.ctx, n_new)                        # n_new: int32 [num_seqs] on the GPU
        t.append(k_new, v_new, k_cache, v_cache)     # rows in sequence order
        t.attention(q, k_cache, v_cache, prefix_table=ids, prefix_len=n, o=o, workspace=ws)
        t.release(done)                              # finished requests' blocks

    ``append_rotary`` rotates queries and keys on the way; ``StepDraft`` adds
    trees of drafted tokens.

    Arrays (int32, device memory): ``block_table`` [num_seqs][max_blocks],
    ``free`` (one bit per block, set = free; all free at first), ``q_start``
    [num_seqs + 1], ``ctx`` [num_seqs] (0 at first), ``position`` and ``slot``
    [max_tokens] (-1 past the step's rows).  Lengths, tables and positions
    count a sequence's own tokens, not the prefix.  A step that does not fit
    is empty and ``device_status`` says why.  The arrays are written in place
    (``t.free.copy_(...)``): the library holds their addresses.  A call with
    ``stream`` does not keep its tensors: they have to live until that stream's
    work is over.
    """

    _HELD = frozenset(("block_table", "free", "q_start", "ctx", "position", "slot", "plan",
                       "status"))

    def __init__(self, config: Config, num_seqs: int, max_blocks: int, max_tokens: int,
                 device="cuda"):
        import torch
        self.config = config
        self.num_seqs, self.max_blocks = int(num_seqs), int(max_blocks)
        self.max_tokens = int(max_tokens)
        for x in (self.num_seqs, self.max_blocks, self.max_tokens):
            _int32(x, "num_seqs, max_blocks and max_tokens")
        ints = int(lib().rbkv_step_plan_ints(self.num_seqs, self.max_tokens))
        if ints == 0 or self.max_blocks < 1 or config.num_blocks < 1:
            raise ValueError("num_seqs, max_blocks, max_tokens and num_blocks must be >= 1")
        words = -(-config.num_blocks // 32)

        def full(value, *shape):
            return torch.full(shape, value, dtype=torch.int32, device=device)

        self.block_table = full(-1, self.num_seqs, self.max_blocks)
        self.free = full(-1, words)
        if config.num_blocks % 32:
            self.free[-1] = (1 << (config.num_blocks % 32)) - 1
        self.q_start, self.ctx = full(0, self.num_seqs + 1), full(0, self.num_seqs)
        self.position, self.slot = full(-1, self.max_tokens), full(-1, self.max_tokens)
        self.plan, self.status = full(0, ints), full(0, 4)
        self.device = self.block_table.device
        self._cfg = config._c()
        self._tables = _StepTables(self.num_seqs, self.max_blocks, self.max_tokens,
                                   *(x.data_ptr() for x in (
                                       self.block_table, self.free, self.q_start, self.ctx,
                                       self.position, self.slot, self.plan, self.status)))
        self._c, self._t = C.byref(self._cfg), C.byref(self._tables)
        self._i32, self._dt = torch.int32, config.torch_dtype
        # (what a call needs, looked up once: a small step takes less time on the
        # GPU than these look-ups do; -2 matches no tensor's device)
        self._index = self.device.index if self.device.type == "cuda" else -2
        self._current, self._raw_stream = _device_calls()
        L = lib()
        self._f_build, self._f_append = L.rbkv_step_build, L.rbkv_step_append
        self._f_attention = L.rbkv_step_attention
        self._f_append_rotary, self._f_draft = L.rbkv_step_append_rotary, \
            L.rbkv_step_attention_draft
        self._table_shape, self._free_shape = self.block_table.shape, self.free.shape
        self._seq_shape = self.ctx.shape
        self._q_shape = torch.Size((self.max_tokens, config.num_heads_q, config.head_dim))
        self._kv_shape = torch.Size((self.max_tokens, config.num_heads_kv, config.head_dim))
        self._cache_shape = torch.Size(config.cache_shape())

    def _ptr(self, t, name, dtype, shape) -> int:
        if t.get_device() == self._index and t.dtype is dtype and t.shape == shape and \
                t.is_contiguous():
            return t.data_ptr()
        if t.device != self.device:
            raise ValueError(f"{name} is on {t.device}, the tables on {self.device}")
        return _dev_ptr(t, name, dtype, shape).value

    def _call(self, fn, *args, stream=None) -> None:
        """A library call on the tables' device (the current one or not)."""
        if self._current() != self._index:
            with _device(self.device):
                return _check(fn(self._c, self._t, *args, _stream(stream)))
        st = self._raw_stream(self._index) if stream is None else _stream(stream)
        status = fn(self._c, self._t, *args, st)
        if status != OK:
            _check(status)

    def build(self, seen, n_new, block_table=None, free=None, stream=None) -> "StepTables":
        """Sequence s holds ``seen[s]`` tokens and takes ``n_new[s]`` more.
        ``block_table`` / ``free``: read from these instead of the tables' own
        (which are written either way)."""
        i32, S = self._i32, self._seq_shape
        self._call(self._f_build, self._ptr(seen, "seen", i32, S),
                   self._ptr(n_new, "n_new", i32, S),
                   None if block_table is None else
                   self._ptr(block_table, "block_table", i32, self._table_shape),
                   None if free is None else self._ptr(free, "free", i32, self._free_shape),
                   stream=stream)
        return self

    def release(self, done, stream=None) -> None:
        """Free the blocks of the sequences with ``done[s] != 0`` (int32)."""
        self._call(lib().rbkv_step_release, self._ptr(done, "done", self._i32, self.ctx.shape),
                   stream=stream)

    def append(self, k_new, v_new, k_cache, v_cache, stream=None) -> None:
        """Scatter the step's K/V rows ([max_tokens][H_kv][D]) into the caches."""
        dt, row, cache = self._dt, self._kv_shape, self._cache_shape
        self._call(self._f_append, self._ptr(k_new, "k_new", dt, row),
                   self._ptr(v_new, "v_new", dt, row), self._ptr(k_cache, "k_cache", dt, cache),
                   self._ptr(v_cache, "v_cache", dt, cache), stream=stream)

    def append_rotary(self, rotary: Rotary, q, k_new, v_new, k_cache, v_cache, q_out=None,
                      prefix_len: int = 0, draft: Optional["StepDraft"] = None, stream=None):
        """``append`` with the rotation on the way, by the positions prefix_len +
        ``position``, or prefix_len + ``draft.place`` (trees need their ``draft``: a kept
        token comes to lie at its place): rotated keys and the values into the caches,
        rotated queries into ``q_out``, which may be ``q`` (rows past the step's are left
        as they were); returns ``q_out``."""
        prefix_len = _int32(int(prefix_len), "prefix_len")
        if q_out is None:
            q_out = _empty_on(stream, self._q_shape, self._dt, self.device)
        dt, row, cache = self._dt, self._kv_shape, self._cache_shape
        self._call(self._f_append_rotary, self._drafted(draft), rotary._on(self.device),
                   prefix_len, self._ptr(q, "q", dt, self._q_shape),
                   self._ptr(q_out, "q_out", dt, self._q_shape),
                   self._ptr(k_new, "k_new", dt, row), self._ptr(v_new, "v_new", dt, row),
                   self._ptr(k_cache, "k_cache", dt, cache),
                   self._ptr(v_cache, "v_cache", dt, cache), stream=stream)
        return q_out

    def _drafted(self, draft):
        if draft is None:
            return None
        if draft.tables is not self:
            raise ValueError("draft belongs to other tables")
        return draft._d

    def workspace_bytes(self, prefix_len: int = 0) -> int:
        prefix_len = _int32(int(prefix_len), "prefix_len")
        with _device(self.device):
            return int(lib().rbkv_step_workspace_bytes(self._c, self._t, prefix_len))

    def attention(self, q, k_cache, v_cache, prefix_table=None, prefix_len: int = 0, o=None,
                  workspace=None, stream=None, draft: Optional["StepDraft"] = None):
        """Every row attends the prefix and its sequence's keys up to its own (with
        ``draft``: those cached before the step, its ancestors' and its own); returns O
        ([max_tokens][H_q][D]; rows past the step's are left as they were)."""
        prefix_len = _int32(int(prefix_len), "prefix_len")
        table = None
        if prefix_table is not None:
            if prefix_table.dim() != 1 or \
                    prefix_table.shape[0] * self.config.block_size < prefix_len:
                raise ValueError("prefix_table must list the blocks of prefix_len tokens")
            table = self._ptr(prefix_table, "prefix_table", self._i32, prefix_table.shape)
        if o is None or workspace is None:
            o, workspace = self._outputs(o, workspace, prefix_len, stream)
        if workspace.get_device() != self._index:
            raise ValueError("workspace is on another device than the tables")
        if not workspace.is_contiguous():
            raise ValueError("workspace must be contiguous")
        dt, cache = self._dt, self._cache_shape
        args = (self._ptr(q, "q", dt, self._q_shape), self._ptr(k_cache, "k_cache", dt, cache),
                self._ptr(v_cache, "v_cache", dt, cache), table, prefix_len,
                self._ptr(o, "o", dt, self._q_shape), workspace.data_ptr(), workspace.nbytes)
        if draft is None:
            self._call(self._f_attention, *args, stream=stream)
        else:
            self._call(self._f_draft, self._drafted(draft), *args, stream=stream)
        return o

    def _outputs(self, o, workspace, prefix_len, stream):
        """O and a workspace where none was given, allocated on the stream that
        uses them."""
        import torch
        if o is None:
            o = _empty_on(stream, self._q_shape, self._dt, self.device)
        if workspace is None:
            workspace = _empty_on(stream, (self.workspace_bytes(prefix_len),), torch.uint8,
                                  self.device)
        return o, workspace

    def device_status(self, stream=None) -> None:
        with _device(self.device):
            _check(lib().rbkv_step_device_status(self._t, _stream(stream)))


class StepDraft(_Arrays):
    """Drafted tokens of a step: a tree of candidate tokens per sequence, attended at
    once, of which one path is kept.  One step of a drafting loop, captured or not::

        d = StepDraft(t)                                  # t: StepTables
        t.build(t.ctx, n_new)                             # new tokens: the trees'
        d.plan(parent)                                    # parent: int32 [max_tokens]
        q = t.append_rotary(rope, q, k_new, v_new, k_cache, v_cache, draft=d)   # per layer
        t.attention(q, k_cache, v_cache, o=o, workspace=ws, draft=d)
        d.accept(tokens, chosen)                          # t.ctx, t.free: cut back
        d.compact(k_cache, v_cache)                       # per layer

    ``parent[r]``: the index, among its sequence's new tokens, of the token that row r
    follows (before its own; -1: none).  Trees have at most 128 tokens; longer runs of
    new tokens are chains, as prompt chunks are.  A bad tree is taken as a chain and
    ``t.device_status`` says so.

    Arrays (int32, device memory, written in place): ``place`` [max_tokens] (position
    of a token once its path is kept; -1 past the rows) and ``ancestors``
    [max_tokens][4] (bit i of word w: the token is, or follows, token 32 w + i) are the
    plan's; ``path`` [max_tokens] (entry q_start[s] + d: row of the d-th kept token of
    sequence s; else -1), ``accepted`` and ``next_token`` [num_seqs] the acceptance's.
    """

    _HELD = frozenset(("place", "ancestors", "path", "accepted", "next_token", "work", "tables"))

    def __init__(self, tables: StepTables):
        import torch
        self.tables = t = tables

        def full(value, *shape):
            return torch.full(shape, value, dtype=torch.int32, device=t.device)

        self.place, self.path = full(-1, t.max_tokens), full(-1, t.max_tokens)
        self.ancestors = full(0, t.max_tokens, 4)
        self.accepted, self.next_token = full(0, t.num_seqs), full(-1, t.num_seqs)
        self.work = full(0, t.num_seqs + 1, 4)
        self._d = C.byref(_StepDraft(*(x.data_ptr() for x in (
            self.place, self.ancestors, self.path, self.accepted, self.next_token, self.work))))
        L = lib()
        self._f_plan, self._f_accept = L.rbkv_step_draft_plan, L.rbkv_step_draft_accept
        self._f_compact = L.rbkv_step_draft_compact
        self._rows = t.position.shape

    def plan(self, parent, stream=None) -> "StepDraft":
        """Work out the trees of the step built last."""
        t = self.tables
        t._call(self._f_plan, self._d, t._ptr(parent, "parent", t._i32, self._rows),
                stream=stream)
        return self

    def accept(self, tokens, chosen, given=None, stream=None) -> "StepDraft":
        """Keep a path of every tree.  ``tokens[r]``: the token of row r; ``chosen[r]``:
        the one chosen to follow it; ``given[s]`` (1 each): leading new tokens of
        sequence s that are not drafted (a prompt chunk: all of them).  From the last
        given token the path goes on to the lowest child that is the chosen token.  Rows
        turned by ``append_rotary(draft=...)``: given tokens have to be a chain, each
        following the one before it (those behind the first that does not are not given,
        and ``t.device_status`` says so).
        Cuts ``t.ctx`` back to the kept tokens and frees the blocks behind them.  Another
        acceptance before the next build, and before ``compact``, takes its place.  A
        sequence released since the build keeps nothing."""
        t, i32 = self.tables, self.tables._i32
        t._call(self._f_accept, self._d, t._ptr(tokens, "tokens", i32, self._rows),
                t._ptr(chosen, "chosen", i32, self._rows),
                None if given is None else t._ptr(given, "given", i32, t._seq_shape),
                stream=stream)
        return self

    def compact(self, k_cache, v_cache, stream=None) -> None:
        """Move the kept tokens' rows of a layer's caches together: once per layer."""
        t = self.tables
        t._call(self._f_compact, self._d, t._ptr(k_cache, "k_cache", t._dt, t._cache_shape),
                t._ptr(v_cache, "v_cache", t._dt, t._cache_shape), stream=stream)


def budget_for_latency(tokens, latency, bound: float) -> int:
    """Largest token count whose latency, interpolated from a measured
    (tokens, latency) profile, stays within ``bound`` (0 if none)."""
    n = len(tokens)
    t = (C.c_int32 * n)(*[int(x) for x in tokens])
    l = (C.c_double * n)(*[float(x) for x in latency])
    r = int(lib().rbkv_budget_for_latency(t, l, n, float(bound)))
    if r < 0:
        raise RbkvError(ERR_INVALID, "bad latency profile")
    return r


def kernel_launches() -> int:
    """Kernels launched through the library by this process so far."""
    return int(lib().rbkv_kernel_launches())


def profile_enable(on: bool = True) -> None:
    lib().rbkv_profile_enable(1 if on else 0)


def profile_reset() -> None:
    lib().rbkv_profile_reset()


def profile_read() -> dict:
    """{kernel: (total_ms, launches)} of the launches timed since the last reset."""
    out = {}
    for name, k in KERNEL_KINDS.items():
        ms, n = C.c_double(), C.c_int64()
        _check(lib().rbkv_profile_read(k, C.byref(ms), C.byref(n)))
        out[name] = (ms.value, n.value)
    return out


GEMM_EPILOGUES = {"plain": 0, "residual": 1, "swiglu": 2}


def gemm_workspace_bytes(m: int, n: int, k: int) -> int:
    """Workspace a GEMM of this size can use to split K (0: it does not)."""
    return int(lib().rbkv_gemm_workspace_bytes(int(m), int(n), int(k)))


def _ws(workspace):
    if workspace is None:
        return _P(None), 0
    return _P(workspace.data_ptr()), workspace.numel() * workspace.element_size()


def gemm(a, b, c=None, residual=None, epilogue: str = "plain", workspace=None, status=None,
         stream=None):
    """C = A B^T (bf16, fp32 accumulation) on the tensor cores with a fused
    epilogue: "plain", "residual" (+ residual) or "swiglu" (B's rows in blocks
    of 128 gate rows and the 128 up rows of the same outputs; C = silu(gate) *
    up).  a: [m][k], b: [n][k]; returns c ([m][n], [m][n/2] for SwiGLU)."""
    import torch
    m, k = a.shape
    n = b.shape[0]
    out_n = n // 2 if epilogue == "swiglu" else n
    if c is None:
        c = torch.empty((m, out_n), dtype=torch.bfloat16, device=a.device)
    dt = torch.bfloat16
    r = _P(None)
    if residual is not None:
        r = _dev_ptr(residual, "residual", dt, (m, n))
    st = _P(status.data_ptr()) if status is not None else _P(None)
    wsp, wsb = _ws(workspace)
    _check(lib().rbkv_gemm_bf16(_dev_ptr(a, "a", dt, (m, k)), _dev_ptr(b, "b", dt, (n, k)),
                                _dev_ptr(c, "c", dt, (m, out_n)), int(m), int(n), int(k), r,
                                GEMM_EPILOGUES[epilogue], wsp, wsb, st, _stream(stream)))
    return c


def gemm_qkv(a, w_qkv, num_heads_q: int, num_heads_kv: int, head_dim: int, out=None,
             workspace=None, status=None, stream=None):
    """The QKV projection in one GEMM: returns Q [m][H_q][D], K and V
    [m][H_kv][D] (contiguous, the attention pass's inputs; written into `out`
    = (q, k, v) when given)."""
    import torch
    m, k = a.shape
    n_q, n_kv = num_heads_q * head_dim, num_heads_kv * head_dim
    dt = torch.bfloat16
    if out is None:
        q = torch.empty((m, num_heads_q, head_dim), dtype=dt, device=a.device)
        kk = torch.empty((m, num_heads_kv, head_dim), dtype=dt, device=a.device)
        vv = torch.empty_like(kk)
    else:
        q, kk, vv = out
    st = _P(status.data_ptr()) if status is not None else _P(None)
    wsp, wsb = _ws(workspace)
    _check(lib().rbkv_gemm_bf16_qkv(_dev_ptr(a, "a", dt, (m, k)),
                                    _dev_ptr(w_qkv, "w_qkv", dt, (n_q + 2 * n_kv, k)),
                                    _dev_ptr(q, "q", dt, (m, num_heads_q, head_dim)),
                                    _dev_ptr(kk, "k", dt, (m, num_heads_kv, head_dim)),
                                    _dev_ptr(vv, "v", dt, (m, num_heads_kv, head_dim)),
                                    int(m), int(n_q), int(n_kv), int(k), wsp, wsb, st,
                                    _stream(stream)))
    return q, kk, vv


def rmsnorm(x, weight, y=None, eps: float = 1e-5, stream=None):
    """RMSNorm of the rows of x ([m][hidden] bf16) with a bf16 weight."""
    import torch
    m, h = x.shape
    if y is None:
        y = torch.empty_like(x)
    dt = torch.bfloat16
    _check(lib().rbkv_rmsnorm_bf16(_dev_ptr(x, "x", dt, (m, h)), _dev_ptr(weight, "weight", dt, (h,)),
                                   _dev_ptr(y, "y", dt, (m, h)), int(m), int(h), float(eps),
                                   _stream(stream)))
    return y


class Router:
    """Routing of requests over independent replicas (host only): the replica
    with the fewest outstanding tokens takes the next request (ties: fewer
    requests held, then the lower index)."""

    def __init__(self, num_replicas: int):
        h = _P()
        _check(lib().rbkv_router_create(int(num_replicas), C.byref(h)))
        self._h = h
        self.num_replicas = int(num_replicas)

    def assign(self, request_id: int, prompt_len: int, output_len: int) -> int:
        out = C.c_int32()
        _check(lib().rbkv_router_assign(self._h, int(request_id), int(prompt_len),
                                        int(output_len), C.byref(out)))
        return int(out.value)

    def progress(self, request_id: int, tokens: int) -> None:
        _check(lib().rbkv_router_progress(self._h, int(request_id), int(tokens)))

    def finish(self, request_id: int) -> None:
        _check(lib().rbkv_router_finish(self._h, int(request_id)))

    def load(self, replica: int) -> int:
        return int(lib().rbkv_router_load(self._h, int(replica)))

    def active(self, replica: int) -> int:
        return int(lib().rbkv_router_active(self._h, int(replica)))

    def close(self) -> None:
        if self._h:
            lib().rbkv_router_destroy(self._h)
            self._h = _P(None)

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


__all__ = ["gemm", "gemm_qkv", "gemm_workspace_bytes", "rmsnorm", "Router", "Frame", "StepTables", "StepDraft", "Rotary", "kv_append_rotary", "budget_for_latency", "seq_states", "SeqStates", "ragged_attention_noalloc", "kernel_launches", "profile_enable", "profile_reset", "profile_read", "Config", "Composer", "Pass", "PassMeta", "kv_append", "ragged_attention",
           "RbkvError", "NoBlocksError", "lib", "library_path", "SIGNATURES"]
