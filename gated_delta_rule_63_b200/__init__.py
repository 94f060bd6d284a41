"""Gated delta-rule layer on NVIDIA B200 (sm_100a): Python binding of libgdr.so.

A thin ctypes layer over the C ABI declared in ``include/gdr.h``: each function
checks dtypes and shapes, passes raw device pointers and the current CUDA
stream, and raises ``GdrError`` on a non-zero status.  Every step of the
computation runs in the library's CUDA kernels; there is no fallback path.
PyTorch is used for device memory and streams only.
"""
from __future__ import annotations

import ctypes
import os
from typing import Optional

import numpy as np

__all__ = [
    "GdrError", "lib", "status_string", "prepare_chunks", "causal_conv", "chunk_prefill",
    "chunk_prefill_noalloc", "chunk_prefill_slots", "prefill_schedule", "prefill_workspace", "linear", "prefill_fused_workspace", "prefill_window",
    "decode_step", "decode_step_slots", "gated_rmsnorm", "get_device_error", "debug_wait_timeout",
    "decay_attn_prefill", "decay_attn_prefill_slots", "decay_attn_workspace",
    "decay_attn_workspace_bound", "decay_attn_decode",
    "decay_attn_decode_slots", "block_norm",
    "HEAD_DIM", "CHUNK",
]

HEAD_DIM = 128
CHUNK = 64
_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libgdr.so")

_vp = ctypes.c_void_p
_ip = ctypes.POINTER(ctypes.c_int32)


class GdrError(RuntimeError):
    def __init__(self, fn: str, code: int):
        detail = lib().gdr_last_error_string().decode() if code == 7 else ""
        super().__init__(f"{fn}: {status_string(code)} (status {code})" + (f" [{detail}]" if detail else ""))
        self.code = code


class FuseArgs(ctypes.Structure):
    """Mirror of ``gdr_prefill_fuse_t``."""
    _fields_ = [("x", _vp), ("conv_w", _vp), ("conv_state_in", _vp), ("conv_state_out", _vp),
                ("z", _vp), ("norm_w", _vp), ("eps", ctypes.c_float), ("y", _vp)]


class BlockNormArgs(ctypes.Structure):
    """Mirror of ``gdr_block_norm_t``."""
    _fields_ = [("x", _vp), ("x_stride", ctypes.c_int64), ("post_norm", ctypes.c_int), ("w_post", _vp),
                ("eps_post", ctypes.c_float), ("gate", _vp), ("gate_stride", ctypes.c_int64),
                ("gate_shared", ctypes.c_int), ("alpha", ctypes.c_float), ("residual", _vp),
                ("residual_stride", ctypes.c_int64), ("residual_fp32", ctypes.c_int), ("residual_out", _vp),
                ("residual_out_stride", ctypes.c_int64), ("w_pre", _vp), ("eps_pre", ctypes.c_float), ("y", _vp),
                ("y_stride", ctypes.c_int64)]


_lib = None


def lib(path: Optional[str] = None):
    """Load libgdr.so (built in-tree by ``gated_delta_rule_63_b200.build``)."""
    global _lib
    if _lib is not None:
        return _lib
    path = path or LIB_PATH
    if not os.path.exists(path):
        raise RuntimeError(f"{path} is missing: build it with `python -m gated_delta_rule_63_b200.build`")
    L = ctypes.CDLL(path)
    L.gdr_status_string.restype = ctypes.c_char_p
    L.gdr_status_string.argtypes = [ctypes.c_int]
    L.gdr_abi_version.restype = ctypes.c_int
    L.gdr_last_error_string.restype = ctypes.c_char_p
    L.gdr_last_error_string.argtypes = []
    L.gdr_prepare_chunks.argtypes = [_ip, ctypes.c_int, ctypes.c_int, _ip, _ip, _ip, ctypes.c_int,
                                     ctypes.POINTER(ctypes.c_int)]
    L.gdr_causal_conv.argtypes = [_vp, _vp, _vp, _vp, _vp, _ip, ctypes.c_int, ctypes.c_int, _vp, _vp]
    L.gdr_chunk_prefill.argtypes = [_vp, _vp, _vp, ctypes.c_int64, ctypes.c_int64, _vp, _vp, _vp,
                                    _vp, ctypes.c_float, ctypes.c_int,
                                    ctypes.c_int, _vp, _ip, ctypes.c_int, _vp, _vp, _vp,
                                    ctypes.POINTER(FuseArgs), _vp, ctypes.c_size_t, _vp]
    L.gdr_chunk_prefill_noalloc.argtypes = [_vp, _vp, _vp, ctypes.c_int64, ctypes.c_int64, _vp, _vp,
                                            _vp, _vp, ctypes.c_float, ctypes.c_int, ctypes.c_int,
                                            _vp, _ip, ctypes.c_int, _vp, _vp, _vp, _vp]
    L.gdr_chunk_prefill_noalloc.restype = ctypes.c_int
    L.gdr_chunk_prefill_noalloc_scratch_bytes.restype = ctypes.c_size_t
    L.gdr_chunk_prefill_noalloc_scratch_bytes.argtypes = []
    L.gdr_chunk_prefill_fused_workspace_size.restype = ctypes.c_size_t
    L.gdr_chunk_prefill_fused_workspace_size.argtypes = [ctypes.c_int] * 6
    L.gdr_chunk_prefill_workspace_size.restype = ctypes.c_size_t
    L.gdr_chunk_prefill_workspace_size.argtypes = [ctypes.c_int, ctypes.c_int, ctypes.c_int,
                                                   ctypes.c_int]
    L.gdr_decode_step.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_float, ctypes.c_int,
                                  ctypes.c_int, _vp, _vp, ctypes.c_int, _vp]
    L.gdr_decode_step_slots.argtypes = [_vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_float, ctypes.c_int,
                                        ctypes.c_int, _vp, ctypes.c_int, _vp, _vp, ctypes.c_int, _vp]
    L.gdr_gated_rmsnorm.argtypes = [_vp, _vp, _vp, ctypes.c_float, ctypes.c_int64, ctypes.c_int, _vp,
                                    _vp]
    L.gdr_get_device_error.argtypes = [ctypes.POINTER(ctypes.c_int), _vp]
    L.gdr_debug_wait_timeout.argtypes = [ctypes.c_int, ctypes.c_ulonglong, _vp, _vp]
    L.gdr_chunk_prefill_slots.argtypes = [_vp, _vp, _vp, ctypes.c_int64, ctypes.c_int64, _vp, _vp, _vp, _vp,
                                          ctypes.c_float, ctypes.c_int, ctypes.c_int, _vp, _ip, ctypes.c_int,
                                          _vp, ctypes.c_int, _vp, ctypes.c_int, _vp, _vp, ctypes.c_size_t, _vp]
    L.gdr_linear.argtypes = [_vp, _vp, _vp, ctypes.c_int64, ctypes.c_int64, ctypes.c_int64, _vp]
    L.gdr_chunk_prefill_schedule.argtypes = [_ip, ctypes.c_int, ctypes.c_int, ctypes.c_size_t, ctypes.c_int,
                                             ctypes.POINTER(ctypes.c_int), ctypes.POINTER(ctypes.c_int)]
    i64 = ctypes.c_int64
    L.gdr_decay_attn_prefill.argtypes = [_vp, _vp, _vp, i64, i64, i64, _vp, ctypes.c_float, ctypes.c_int,
                                         ctypes.c_int, _vp, _vp, ctypes.c_int, _vp, _vp, _vp, _vp, ctypes.c_size_t,
                                         _vp]
    L.gdr_decay_attn_prefill_slots.argtypes = [_vp, _vp, _vp, i64, i64, i64, _vp, ctypes.c_float, ctypes.c_int,
                                               ctypes.c_int, _vp, _vp, ctypes.c_int, _vp, ctypes.c_int, _vp,
                                               ctypes.c_int, _vp, _vp, ctypes.c_size_t, _vp]
    L.gdr_decay_attn_decode.argtypes = [_vp, _vp, _vp, i64, i64, i64, _vp, ctypes.c_float, ctypes.c_int,
                                        ctypes.c_int, _vp, _vp, ctypes.c_int, _vp]
    L.gdr_decay_attn_decode_slots.argtypes = [_vp, _vp, _vp, i64, i64, i64, _vp, ctypes.c_float, ctypes.c_int,
                                              ctypes.c_int, _vp, ctypes.c_int, _vp, _vp, ctypes.c_int, _vp]
    L.gdr_decay_attn_prefill_workspace_size.restype = ctypes.c_size_t
    L.gdr_decay_attn_prefill_workspace_size.argtypes = [_vp, ctypes.c_int, ctypes.c_int]
    L.gdr_decay_attn_prefill_workspace_bound.restype = ctypes.c_size_t
    L.gdr_decay_attn_prefill_workspace_bound.argtypes = [i64, ctypes.c_int, ctypes.c_int]
    L.gdr_block_norm.argtypes = [ctypes.POINTER(BlockNormArgs), i64, i64, _vp]
    for fn in ("gdr_decay_attn_prefill", "gdr_decay_attn_prefill_slots", "gdr_decay_attn_decode",
               "gdr_decay_attn_decode_slots", "gdr_block_norm"):
        getattr(L, fn).restype = ctypes.c_int
    for fn in ("gdr_prepare_chunks", "gdr_causal_conv", "gdr_chunk_prefill", "gdr_decode_step",
               "gdr_decode_step_slots", "gdr_gated_rmsnorm", "gdr_get_device_error",
               "gdr_debug_wait_timeout", "gdr_chunk_prefill_slots", "gdr_chunk_prefill_schedule", "gdr_linear"):
        getattr(L, fn).restype = ctypes.c_int
    _lib = L
    return L


def status_string(code: int) -> str:
    return lib().gdr_status_string(int(code)).decode()


def _check(fn: str, code: int):
    if code != 0:
        raise GdrError(fn, code)


# ---------------------------------------------------------------------------
# marshalling helpers
# ---------------------------------------------------------------------------

_torch_module = None


def _torch():
    global _torch_module
    if _torch_module is None:
        import torch
        _torch_module = torch
    return _torch_module


def _ptr(t, dtype=None, name="tensor", rows=False):
    """Device pointer of a tensor; with rows=True only the last two dims must be dense."""
    if t is None:
        return None
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if rows:
        if t.dim() != 3 or t.stride(2) != 1 or t.stride(1) != t.shape[2]:
            raise ValueError(f"{name} must be [T, heads, 128] with dense rows")
    elif not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t.data_ptr()


def _tok_stride(t):
    return 0 if t is None else int(t.stride(0))


def _device_of(*tensors):
    """The one device of the given tensors (None skipped); tensors on two devices raise.

    Each call runs on that device with its stream, so no kernel is handed a pointer into
    another GPU's memory."""
    dev = None
    for t in tensors:
        d = getattr(t, "device", None)
        if d is None or d.type != "cuda":
            continue   # not a CUDA tensor: _ptr rejects it by name
        if dev is None:
            dev = d
        elif d != dev:
            raise ValueError(f"tensors on {dev} and {d}: all tensors of a call must be on one device")
    return dev


def _stream(stream=None, device=None):
    torch = _torch()
    if stream is None:
        return torch.cuda.current_stream(device).cuda_stream
    if device is not None and getattr(stream, "device", device) != device:
        raise ValueError(f"stream on {stream.device}, tensors on {device}")
    return stream.cuda_stream


def _host_cu(cu_host):
    cu = np.ascontiguousarray(np.asarray(cu_host), dtype=np.int32)
    return cu, cu.ctypes.data_as(_ip)


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------

def prepare_chunks(cu_seqlens_host, chunk: int = CHUNK):
    """Chunk table (chunk_seq, chunk_start, chunk_len) of packed sequences."""
    cu, cup = _host_cu(cu_seqlens_host)
    n = cu.shape[0] - 1
    total = int(cu[-1]) if n > 0 else 0
    cap = max(1, total // max(chunk, 1) + n + 1)
    seq = np.zeros(cap, np.int32); st = np.zeros(cap, np.int32); ln = np.zeros(cap, np.int32)
    m = ctypes.c_int(0)
    _check("gdr_prepare_chunks", lib().gdr_prepare_chunks(
        cup, n, int(chunk), seq.ctypes.data_as(_ip), st.ctypes.data_as(_ip), ln.ctypes.data_as(_ip),
        cap, ctypes.byref(m)))
    k = m.value
    return seq[:k].copy(), st[:k].copy(), ln[:k].copy()


def causal_conv(x, w, cu_seqlens, cu_seqlens_host, conv_state_in=None, conv_state_out=None, y=None,
                stream=None):
    """Depthwise causal conv4 + SiLU.  x [T, C] bf16, w [C, 4] bf16 -> y [T, C] bf16."""
    torch = _torch()
    bf = torch.bfloat16
    cu, cup = _host_cu(cu_seqlens_host)
    if y is None:
        y = torch.empty_like(x)
    C = x.shape[1]
    dev = _device_of(x, w, conv_state_in, conv_state_out, cu_seqlens, y)
    with torch.cuda.device(dev):
        _check("gdr_causal_conv", lib().gdr_causal_conv(
            _ptr(x, bf, "x"), _ptr(w, bf, "w"), _ptr(conv_state_in, bf, "conv_state_in"),
            _ptr(conv_state_out, bf, "conv_state_out"), _ptr(cu_seqlens, torch.int32, "cu_seqlens"), cup,
            cu.shape[0] - 1, C, _ptr(y, bf, "y"), _stream(stream, dev)))
    return y


DEFAULT_WORKSPACE_BYTES = 512 << 20


def prefill_window(cu_seqlens_host, hv: int, max_bytes: int = DEFAULT_WORKSPACE_BYTES,
                   has_final_state: bool = True) -> int:
    """Largest chunk window (<= the longest sequence) whose workspace fits max_bytes."""
    cu = np.asarray(cu_seqlens_host, dtype=np.int64)
    n = len(cu) - 1
    if n <= 0:
        return 1
    max_chunks = int(max(1, ((np.diff(cu) + CHUNK - 1) // CHUNK).max()))
    per_chunk = lib().gdr_chunk_prefill_workspace_size(n, hv, 1, 1)
    carry = lib().gdr_chunk_prefill_workspace_size(n, hv, 1, int(has_final_state)) - per_chunk
    fit = max(1, (max_bytes - carry) // per_chunk)
    return int(min(max_chunks, fit))


def prefill_schedule(cu_seqlens_host, hv: int, workspace_bytes: int, has_final_state: bool = True):
    """(windows, pipelined) of gdr_chunk_prefill for these sequences and workspace size on the
    current CUDA device: the number of windows (one operand launch and one state launch each)
    and whether the next window is built beside the current one's state walk."""
    cu, cup = _host_cu(cu_seqlens_host)
    w, pl = ctypes.c_int(0), ctypes.c_int(0)
    _check("gdr_chunk_prefill_schedule", lib().gdr_chunk_prefill_schedule(
        cup, cu.shape[0] - 1, int(hv), int(workspace_bytes), int(bool(has_final_state)), ctypes.byref(w),
        ctypes.byref(pl)))
    return w.value, bool(pl.value)


def prefill_workspace(cu_seqlens_host, hv: int, device, window: Optional[int] = None,
                      has_final_state: bool = True):
    """A torch uint8 device buffer sized for gdr_chunk_prefill."""
    torch = _torch()
    cu = np.asarray(cu_seqlens_host)
    n = len(cu) - 1
    if window is None:
        window = prefill_window(cu_seqlens_host, hv, has_final_state=has_final_state)
    nbytes = lib().gdr_chunk_prefill_workspace_size(max(n, 1), hv, max(int(window), 1),
                                                    int(has_final_state))
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def prefill_fused_workspace(cu_seqlens_host, hk: int, hv: int, device, window: Optional[int] = None,
                            has_final_state: bool = True):
    """Workspace for gdr_chunk_prefill running the conv in the same call: the conv output, then the records."""
    torch = _torch()
    cu = np.asarray(cu_seqlens_host)
    n = len(cu) - 1
    T = int(cu[-1]) if n > 0 else 0
    if window is None:
        window = prefill_window(cu_seqlens_host, hv, has_final_state=has_final_state)
    nbytes = lib().gdr_chunk_prefill_fused_workspace_size(max(n, 1), int(hk), int(hv), T, max(int(window), 1),
                                                          int(has_final_state))
    return torch.empty(max(int(nbytes), 16), dtype=torch.uint8, device=device)


def chunk_prefill(q, k, v, a, b, A_log, dt_bias, cu_seqlens, cu_seqlens_host, h0=None, hT=None,
                  o=None, scale: float = 1.0, fuse: Optional[dict] = None, workspace=None,
                  window: Optional[int] = None, stream=None):
    """Chunk-64 prefill.  q, k [T, hk, 128], v [T, hv, 128], a, b [T, hv] bf16.

    q, k, v may be token-strided views (e.g. slices of the [T, q|k|v] conv output); with the
    conv run by the same call (``fuse`` holding "x", "conv_w" and "hk") they are None.

    Returns o [T, hv, 128] bf16 (and writes hT [N, hv, 128, 128] fp32 when given).
    ``fuse`` (optional) maps gdr_prefill_fuse_t field names to tensors.
    """
    torch = _torch()
    bf, f32 = torch.bfloat16, torch.float32
    cu, cup = _host_cu(cu_seqlens_host)
    fz = None
    if fuse is not None:
        fz = FuseArgs()
        for name in ("x", "conv_w", "conv_state_in", "conv_state_out", "z", "y"):
            setattr(fz, name, _ptr(fuse.get(name), bf, name))
        fz.norm_w = _ptr(fuse.get("norm_w"), f32, "norm_w")
        fz.eps = float(fuse.get("eps", 1e-6))
    hk = q.shape[1] if q is not None else int(fuse["hk"])
    hv = a.shape[1]
    if q is not None and k.stride(0) != q.stride(0):
        raise ValueError("q and k must share their token stride")
    if o is None and (fuse is None or fuse.get("y") is None or fuse.get("keep_o", False)):
        T = a.shape[0]
        o = torch.empty((T, hv, HEAD_DIM), dtype=bf, device=a.device)
    if workspace is None:
        if fuse is not None and fuse.get("x") is not None:
            workspace = prefill_fused_workspace(cu_seqlens_host, hk, hv, a.device, window, hT is not None)
        else:
            workspace = prefill_workspace(cu_seqlens_host, hv, a.device, window, hT is not None)
    fuse_tensors = [fuse.get(n) for n in ("x", "conv_w", "conv_state_in", "conv_state_out", "z", "y",
                                          "norm_w")] if fuse is not None else []
    dev = _device_of(q, k, v, a, b, A_log, dt_bias, cu_seqlens, h0, hT, o, workspace, *fuse_tensors)
    with torch.cuda.device(dev):
        _check("gdr_chunk_prefill", lib().gdr_chunk_prefill(
            _ptr(q, bf, "q", rows=True), _ptr(k, bf, "k", rows=True), _ptr(v, bf, "v", rows=True),
            _tok_stride(q), _tok_stride(v), _ptr(a, bf, "a"), _ptr(b, bf, "b"),
            _ptr(A_log, f32, "A_log"), _ptr(dt_bias, f32, "dt_bias"), float(scale), int(hk), int(hv),
            _ptr(cu_seqlens, torch.int32, "cu_seqlens"), cup, cu.shape[0] - 1,
            _ptr(h0, f32, "h0"), _ptr(hT, f32, "hT"), _ptr(o, bf, "o"),
            ctypes.byref(fz) if fz is not None else None, _ptr(workspace, torch.uint8, "workspace"),
            int(workspace.numel()), _stream(stream, dev)))
    return o


def chunk_prefill_noalloc(q, k, v, a, b, A_log, dt_bias, cu_seqlens, cu_seqlens_host, h0=None,
                          hT=None, o=None, scale: float = 1.0, stream=None):
    """gdr_chunk_prefill on the library's own scratch array (no workspace argument).

    For callers that cannot allocate device memory; see gdr_chunk_prefill_noalloc
    in include/gdr.h for the size limit and the rule that calls must not overlap.
    """
    torch = _torch()
    bf, f32 = torch.bfloat16, torch.float32
    cu, cup = _host_cu(cu_seqlens_host)
    hv = a.shape[1]
    if o is None:
        o = torch.empty((a.shape[0], hv, HEAD_DIM), dtype=bf, device=a.device)
    dev = _device_of(q, k, v, a, b, A_log, dt_bias, cu_seqlens, h0, hT, o)
    with torch.cuda.device(dev):
        _check("gdr_chunk_prefill_noalloc", lib().gdr_chunk_prefill_noalloc(
            _ptr(q, bf, "q", rows=True), _ptr(k, bf, "k", rows=True), _ptr(v, bf, "v", rows=True),
            _tok_stride(q), _tok_stride(v), _ptr(a, bf, "a"), _ptr(b, bf, "b"),
            _ptr(A_log, f32, "A_log"), _ptr(dt_bias, f32, "dt_bias"), float(scale), int(q.shape[1]),
            int(hv), _ptr(cu_seqlens, torch.int32, "cu_seqlens"), cup, cu.shape[0] - 1,
            _ptr(h0, f32, "h0"), _ptr(hT, f32, "hT"), _ptr(o, bf, "o"), _stream(stream, dev)))
    return o


def chunk_prefill_slots(q, k, v, a, b, A_log, dt_bias, cu_seqlens, cu_seqlens_host, state_pool, slot,
                        init_from_pool: bool = False, o=None, scale: float = 1.0, workspace=None, stream=None):
    """gdr_chunk_prefill on a pool of cached states: sequence n starts from entry slot[n] of
    state_pool (or from zero, init_from_pool=False) and leaves its final state there.  A slot
    outside the pool is a sequence that starts from zero and keeps no state."""
    torch = _torch()
    bf, f32 = torch.bfloat16, torch.float32
    cu, cup = _host_cu(cu_seqlens_host)
    hv = a.shape[1]
    if o is None:
        o = torch.empty((a.shape[0], hv, HEAD_DIM), dtype=bf, device=a.device)
    if workspace is None:
        workspace = prefill_workspace(cu, hv, a.device, has_final_state=False)
    dev = _device_of(q, k, v, a, b, A_log, dt_bias, cu_seqlens, state_pool, slot, o, workspace)
    with torch.cuda.device(dev):
        _check("gdr_chunk_prefill_slots", lib().gdr_chunk_prefill_slots(
            _ptr(q, bf, "q", rows=True), _ptr(k, bf, "k", rows=True), _ptr(v, bf, "v", rows=True),
            _tok_stride(q), _tok_stride(v), _ptr(a, bf, "a"), _ptr(b, bf, "b"),
            _ptr(A_log, f32, "A_log"), _ptr(dt_bias, f32, "dt_bias"), float(scale), int(q.shape[1]),
            int(hv), _ptr(cu_seqlens, torch.int32, "cu_seqlens"), cup, cu.shape[0] - 1,
            _ptr(state_pool, f32, "state_pool"), int(state_pool.shape[0]), _ptr(slot, torch.int32, "slot"),
            int(bool(init_from_pool)), _ptr(o, bf, "o"), _ptr(workspace, torch.uint8, "workspace"),
            workspace.numel(), _stream(stream, dev)))
    return o


def decode_step(x, conv_w, conv_state, a, b, A_log, dt_bias, state, o=None, scale: float = 1.0,
                hk: int = 16, stream=None):
    """One token for each of B sequences; conv_state and state are updated in place."""
    torch = _torch()
    bf, f32 = torch.bfloat16, torch.float32
    B, hv = a.shape
    if o is None:
        o = torch.empty((B, hv, HEAD_DIM), dtype=bf, device=a.device)
    dev = _device_of(x, conv_w, conv_state, a, b, A_log, dt_bias, state, o)
    with torch.cuda.device(dev):
        _check("gdr_decode_step", lib().gdr_decode_step(
            _ptr(x, bf, "x"), _ptr(conv_w, bf, "conv_w"), _ptr(conv_state, bf, "conv_state"),
            _ptr(a, bf, "a"), _ptr(b, bf, "b"), _ptr(A_log, f32, "A_log"), _ptr(dt_bias, f32, "dt_bias"),
            float(scale), int(hk), int(hv), _ptr(state, f32, "state"), _ptr(o, bf, "o"), int(B),
            _stream(stream, dev)))
    return o


def decode_step_slots(x, conv_w, conv_state_pool, a, b, A_log, dt_bias, state_pool, slot, o=None,
                      scale: float = 1.0, hk: int = 16, stream=None):
    """One token for each of B rows; row i updates pool entry slot[i] of both pools in place.

    slot is an int32 CUDA tensor [B]; a slot outside [0, n_slots) is a padding row (zero o).
    """
    torch = _torch()
    bf, f32 = torch.bfloat16, torch.float32
    B, hv = a.shape
    n_slots = int(state_pool.shape[0])
    if tuple(slot.shape) != (B,):
        raise ValueError(f"slot must have shape ({B},), got {tuple(slot.shape)}")
    if int(conv_state_pool.shape[0]) != n_slots:
        raise ValueError("conv_state_pool and state_pool must hold the same number of slots")
    if o is None:
        o = torch.empty((B, hv, HEAD_DIM), dtype=bf, device=a.device)
    dev = _device_of(x, conv_w, conv_state_pool, a, b, A_log, dt_bias, state_pool, slot, o)
    with torch.cuda.device(dev):
        _check("gdr_decode_step_slots", lib().gdr_decode_step_slots(
            _ptr(x, bf, "x"), _ptr(conv_w, bf, "conv_w"), _ptr(conv_state_pool, bf, "conv_state_pool"),
            _ptr(a, bf, "a"), _ptr(b, bf, "b"), _ptr(A_log, f32, "A_log"), _ptr(dt_bias, f32, "dt_bias"),
            float(scale), int(hk), int(hv), _ptr(state_pool, f32, "state_pool"), n_slots,
            _ptr(slot, torch.int32, "slot"), _ptr(o, bf, "o"), int(B), _stream(stream, dev)))
    return o


def linear(x, w, y=None, stream=None):
    """y = x w^T: x [M, K], w [N, K] bf16 CUDA tensors (dense rows) -> y [M, N] bf16."""
    torch = _torch()
    bf = torch.bfloat16
    if x.dim() != 2 or w.dim() != 2 or x.shape[1] != w.shape[1]:
        raise ValueError("linear: x [M, K] and w [N, K] with the same K")
    M, K = x.shape
    N = w.shape[0]
    if y is None:
        y = torch.empty((M, N), dtype=bf, device=x.device)
    if tuple(y.shape) != (M, N):
        raise ValueError("linear: y must be [M, N]")
    dev = _device_of(x, w, y)
    with torch.cuda.device(dev):
        _check("gdr_linear", lib().gdr_linear(_ptr(x, bf, "x"), _ptr(w, bf, "w"), _ptr(y, bf, "y"), int(M), int(N),
                                              int(K), _stream(stream, dev)))
    return y


# The calls below are short enough on the device for the marshalling to show: one pass over the
# tensors, the device entered only when it is not the current one.

class _Call:
    """Device and stream of a call, taken from its first tensor; every other must be there too."""
    __slots__ = ("torch", "tensor", "index")

    def __init__(self, t, name):
        self.torch = torch = _torch()
        self.tensor = torch.Tensor
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        self.index = t.get_device()   # -1 for the host
        if self.index < 0 or not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")

    def refuse(self, t, dtype, name):
        """What is wrong with a tensor's type, dtype or device."""
        if not isinstance(t, self.tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype is not dtype:
            raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
        if not t.is_cuda:
            raise ValueError(f"{name} must be a CUDA tensor")
        raise ValueError(f"tensors on cuda:{self.index} and {t.device}: all tensors of a call must be on one device")

    def dense(self, t, dtype, name, shape):
        """Pointer of a contiguous tensor of that shape (None passes)."""
        if t is None:
            return None
        if not isinstance(t, self.tensor) or t.dtype is not dtype or t.get_device() != self.index:
            self.refuse(t, dtype, name)
        if t.shape != shape:
            raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
        if not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous")
        return t.data_ptr()

    def heads(self, t, name, rows, heads):
        """(pointer, token stride) of a bf16 [>= rows, heads, 128] tensor whose last two dims are dense."""
        bf16 = self.torch.bfloat16
        if not isinstance(t, self.tensor) or t.dtype is not bf16 or t.get_device() != self.index:
            self.refuse(t, bf16, name)
        shape = t.shape
        if len(shape) != 3 or shape[2] != HEAD_DIM or shape[1] != heads or shape[0] < rows:
            raise ValueError(f"{name} must be [{rows}, {heads}, {HEAD_DIM}], got {tuple(shape)}")
        if t.is_contiguous():
            return t.data_ptr(), 0
        st = t.stride()
        if st[2] != 1 or (heads > 1 and st[1] != HEAD_DIM) or st[0] < heads * HEAD_DIM:
            raise ValueError(f"{name} must be [T, heads, 128] with dense rows that do not overlap")
        return t.data_ptr(), st[0]

    def rows(self, t, dtype, name, rows, d):
        """(pointer, row stride) of `rows` rows of d values: contiguous, or [rows, d] with dense rows."""
        if t is None:
            return None, 0
        if not isinstance(t, self.tensor) or t.dtype is not dtype or t.get_device() != self.index:
            self.refuse(t, dtype, name)
        if t.numel() != rows * d or t.shape[-1] != d:
            raise ValueError(f"{name} must hold {rows} rows of {d} values, got {tuple(t.shape)}")
        if t.is_contiguous():
            return t.data_ptr(), 0
        if t.dim() != 2 or t.stride(1) != 1 or t.stride(0) < d:
            raise ValueError(f"{name} must be contiguous, or [rows, d] with dense rows that do not overlap")
        return t.data_ptr(), t.stride(0)

    def run(self, name, fn, stream, *args):
        """fn(*args, stream) on the call's device."""
        cuda, index = self.torch.cuda, self.index
        if stream is None:
            handle = _current_stream(index)
        else:
            if getattr(stream, "device", None) is not None and stream.device.index != index:
                raise ValueError(f"stream on {stream.device}, tensors on cuda:{index}")
            handle = stream.cuda_stream
        if cuda.current_device() == index:
            code = fn(*args, handle)
        else:
            with cuda.device(index):
                code = fn(*args, handle)
        if code != 0:
            raise GdrError(name, code)


def _current_stream(index):
    """Handle of the current stream of a device: torch's own short way where it has one (making the
    Stream object takes 1.2 us, a tenth of a short call)."""
    torch = _torch()
    raw = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    return raw(index) if raw is not None else torch.cuda.current_stream(index).cuda_stream


def _on_stream(stream, make):
    """make() with the tensors it makes belonging to the call's stream: given back to the allocator
    (a workspace at the end of the call), their memory is then not used before the call's kernels
    are through with it."""
    if stream is None:
        return make()
    with _torch().cuda.stream(stream):
        return make()


def _decay_inputs(q, k, v, log_decay, rows):
    """The call and the checked arguments the decayed linear attention calls share, in the ABI's order."""
    call = _Call(q, "q")
    if q.dim() != 3 or v.dim() != 3:
        raise ValueError("q and v must be [T, heads, 128]")
    hk, hv = int(q.shape[1]), int(v.shape[1])
    qp, qs = call.heads(q, "q", rows, hk)
    kp, ks = call.heads(k, "k", rows, hk)
    vp, vs = call.heads(v, "v", rows, hv)
    return call, (qp, kp, vp, qs, ks, vs, call.dense(log_decay, _torch().float32, "log_decay", (hv,))), hk, hv


def _decay_o(call, o, v, hv, rows, stream):
    """o (made when None) and its pointer; it may have more rows than the call writes."""
    torch = _torch()
    if o is None:
        # v's shape, dense (v has dense rows)
        o = torch.empty_like(v) if stream is None else _on_stream(stream, lambda: torch.empty_like(v))
        return o, o.data_ptr()
    if isinstance(o, torch.Tensor) and (o.dim() != 3 or o.shape[0] < rows):
        raise ValueError(f"o must be [{rows}, {hv}, {HEAD_DIM}], got {tuple(o.shape)}")
    return o, call.dense(o, torch.bfloat16, "o", (o.shape[0], hv, HEAD_DIM))


def decay_attn_workspace(cu_seqlens_host, hv: int, device):
    """A torch uint8 device buffer sized for gdr_decay_attn_prefill, or None when it needs none."""
    torch = _torch()
    cu, _ = _host_cu(cu_seqlens_host)
    nbytes = int(lib().gdr_decay_attn_prefill_workspace_size(cu.ctypes.data, cu.shape[0] - 1, int(hv)))
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def decay_attn_workspace_bound(max_tokens: int, max_seqs: int, hv: int, device):
    """A torch uint8 device buffer that is enough for every decayed-attention prefill of at most
    max_seqs sequences with max_tokens tokens together (the need of one call may exceed that of a
    longer one), or None when none of them needs one."""
    torch = _torch()
    nbytes = int(lib().gdr_decay_attn_prefill_workspace_bound(int(max_tokens), int(max_seqs), int(hv)))
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def _decay_prefill(name, q, k, v, log_decay, cu_seqlens, cu_seqlens_host, states, o, scale, workspace, stream):
    """The prefill call `name`; states(call, n, hv) gives its arguments between n_seqs and o."""
    torch = _torch()
    cu = np.ascontiguousarray(cu_seqlens_host, dtype=np.int32)
    cup = cu.ctypes.data
    if cu.ndim != 1 or cu.shape[0] < 1:
        raise ValueError("cu_seqlens_host must hold n_seqs + 1 offsets")
    n, total = cu.shape[0] - 1, int(cu[-1])
    call, ins, hk, hv = _decay_inputs(q, k, v, log_decay, total)
    o, op = _decay_o(call, o, v, hv, total, stream)
    if workspace is None:
        need = lib().gdr_decay_attn_prefill_workspace_size(cup, n, hv)
        if need:
            workspace = _on_stream(stream, lambda: torch.empty(need, dtype=torch.uint8, device=v.device))
    wp, wbytes = (None, 0) if workspace is None else (
        call.dense(workspace, torch.uint8, "workspace", workspace.shape), workspace.numel())
    call.run(name, getattr(lib(), name), stream, *ins, float(scale), hk, hv,
             call.dense(cu_seqlens, torch.int32, "cu_seqlens", cu.shape), cup, n, *states(call, n, hv), op, wp, wbytes)
    return o


def decay_attn_prefill(q, k, v, log_decay, cu_seqlens, cu_seqlens_host, h0=None, hT=None, o=None,
                       scale: float = 1.0, workspace=None, stream=None):
    """Decayed linear attention over packed sequences: H_t = exp(log_decay) H_{t-1} + k_t v_t^T,
    o_t = scale H_t^T q_t.  q, k [T, hk, 128], v [T, hv, 128] bf16 (token-strided views allowed),
    log_decay [hv] fp32.  Returns o [T, hv, 128] bf16 (and writes hT [N, hv, 128, 128] fp32 when
    given); rows of o behind the last sequence are left as they were.  Without a workspace one is
    made for the call when it needs one (decay_attn_workspace); calls that may run at the same time
    must not share one."""
    f32 = _torch().float32

    def states(call, n, hv):
        shape = (n, hv, HEAD_DIM, HEAD_DIM)
        return call.dense(h0, f32, "h0", shape), call.dense(hT, f32, "hT", shape)
    return _decay_prefill("gdr_decay_attn_prefill", q, k, v, log_decay, cu_seqlens, cu_seqlens_host, states, o, scale,
                          workspace, stream)


def decay_attn_prefill_slots(q, k, v, log_decay, cu_seqlens, cu_seqlens_host, state_pool, slot,
                             init_from_pool: bool = False, o=None, scale: float = 1.0, workspace=None,
                             stream=None):
    """decay_attn_prefill on a pool of cached states: sequence n starts from entry slot[n] of
    state_pool (or from zero, init_from_pool=False) and leaves its final state there.  A slot
    outside the pool is a sequence that starts from zero and keeps no state."""
    torch = _torch()
    n_slots = int(state_pool.shape[0])

    def states(call, n, hv):
        return (call.dense(state_pool, torch.float32, "state_pool", (n_slots, hv, HEAD_DIM, HEAD_DIM)), n_slots,
                call.dense(slot, torch.int32, "slot", (n,)), int(bool(init_from_pool)))
    return _decay_prefill("gdr_decay_attn_prefill_slots", q, k, v, log_decay, cu_seqlens, cu_seqlens_host, states, o,
                          scale, workspace, stream)


def decay_attn_decode(q, k, v, log_decay, state, o=None, scale: float = 1.0, stream=None):
    """One token of decayed linear attention for each of B sequences; q, k [B, hk, 128],
    v [B, hv, 128] bf16, state [B, hv, 128, 128] fp32 updated in place -> o [B, hv, 128] bf16."""
    B = int(v.shape[0])
    call, ins, hk, hv = _decay_inputs(q, k, v, log_decay, B)
    o, op = _decay_o(call, o, v, hv, B, stream)
    call.run("gdr_decay_attn_decode", lib().gdr_decay_attn_decode, stream, *ins, float(scale), hk, hv,
             call.dense(state, _torch().float32, "state", (B, hv, HEAD_DIM, HEAD_DIM)), op, B)
    return o


def decay_attn_decode_slots(q, k, v, log_decay, state_pool, slot, o=None, scale: float = 1.0, stream=None):
    """decay_attn_decode on a pool of cached states: row i updates entry slot[i] in place; a slot
    outside the pool is a padding row (zero o)."""
    torch = _torch()
    B, n_slots = int(v.shape[0]), int(state_pool.shape[0])
    call, ins, hk, hv = _decay_inputs(q, k, v, log_decay, B)
    o, op = _decay_o(call, o, v, hv, B, stream)
    call.run("gdr_decay_attn_decode_slots", lib().gdr_decay_attn_decode_slots, stream, *ins, float(scale), hk, hv,
             call.dense(state_pool, torch.float32, "state_pool", (n_slots, hv, HEAD_DIM, HEAD_DIM)), n_slots,
             call.dense(slot, torch.int32, "slot", (B,)), op, B)
    return o


def block_norm(x, residual=None, gate=None, post_norm: bool = False, w_post=None, w_pre=None, alpha: float = 1.0,
               eps: float = 1e-6, eps_post: Optional[float] = None, residual_out=None, y=None,
               want_residual: bool = True, want_y: bool = True, stream=None):
    """The norms after and before a block with its gate and residual, row by row:
    u = x / rms(x) * w_post (post_norm) or x, r = residual + alpha * gate * u,
    y = r / rms(r) * w_pre.  x, y bf16 [..., d]; gate bf16 [d] or like x; residual and
    residual_out bf16 or fp32 (like each other).  Returns (residual_out, y); residual_out may be
    residual and y may be x (in place).  want_residual / want_y = False leaves that output out
    (None) when no tensor is given for it."""
    torch = _torch()
    bf, f32 = torch.bfloat16, torch.float32
    call = _Call(x, "x")
    d = x.shape[-1] if x.dim() else 0
    rows = x.numel() // d if d else 0
    xp, xs = call.rows(x, bf, "x", rows, d)
    rdt = residual.dtype if residual is not None else residual_out.dtype if residual_out is not None else bf
    if rdt is not bf and rdt is not f32:
        raise TypeError(f"residual must be torch.bfloat16 or torch.float32, got {rdt}")
    shared = gate is not None and gate.dim() == 1
    gp, gs = call.rows(gate, bf, "gate", 1 if shared else rows, d)
    rp, rs = call.rows(residual, rdt, "residual", rows, d)
    if residual_out is None and want_residual:   # (x's shape, dense)
        make = (lambda: torch.empty_like(x)) if rdt is bf else (lambda: torch.empty_like(x, dtype=rdt))
        residual_out = make() if stream is None else _on_stream(stream, make)
        op, os_ = residual_out.data_ptr(), 0
    else:
        op, os_ = call.rows(residual_out, rdt, "residual_out", rows, d)
    if y is None and want_y:
        y = torch.empty_like(x) if stream is None else _on_stream(stream, lambda: torch.empty_like(x))
        yp, ys = y.data_ptr(), 0
    else:
        yp, ys = call.rows(y, bf, "y", rows, d)
    args = BlockNormArgs(xp, xs, 1 if post_norm else 0, call.dense(w_post, f32, "w_post", (d,)),
                         eps if eps_post is None else eps_post, gp, gs, 1 if shared else 0, alpha, rp, rs,
                         1 if rdt == f32 else 0, op, os_, call.dense(w_pre, f32, "w_pre", (d,)), eps, yp, ys)
    call.run("gdr_block_norm", lib().gdr_block_norm, stream, ctypes.byref(args), rows, d)
    return residual_out, y


def gated_rmsnorm(o, z, w=None, eps: float = 1e-6, y=None, stream=None):
    """y = o / sqrt(mean(o^2) + eps) * w * SiLU(z) over rows of 128."""
    torch = _torch()
    bf = torch.bfloat16
    if y is None:
        y = torch.empty_like(o)
    d = o.shape[-1]
    rows = o.numel() // d
    dev = _device_of(o, z, w, y)
    with torch.cuda.device(dev):
        _check("gdr_gated_rmsnorm", lib().gdr_gated_rmsnorm(
            _ptr(o, bf, "o"), _ptr(z, bf, "z"), _ptr(w, torch.float32, "w"), float(eps), int(rows), int(d),
            _ptr(y, bf, "y"), _stream(stream, dev)))
    return y


def get_device_error(stream=None) -> int:
    """Read and clear the library's device error word (synchronises the stream)."""
    v = ctypes.c_int(0)
    _check("gdr_get_device_error", lib().gdr_get_device_error(ctypes.byref(v), _stream(stream)))
    return v.value


def debug_wait_timeout(kind: int, limit: int, device=None, stream=None) -> int:
    """Run the bounded-wait self-test kernel (gdr_debug_wait_timeout): one CTA waits on an
    mbarrier nothing arrives at until `limit` runs out (kind 0: polls, kind 1: SM cycles).
    Returns the kernel's own verdict (0 = the wait gave up); the device error word then holds
    GDR_ERR_TIMEOUT (read it with get_device_error)."""
    torch = _torch()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    with torch.cuda.device(dev):
        res = torch.full((1,), -1, dtype=torch.int32, device=dev)
        _check("gdr_debug_wait_timeout", lib().gdr_debug_wait_timeout(int(kind), int(limit), res.data_ptr(),
                                                                      _stream(stream, dev)))
        return int(res.item())
