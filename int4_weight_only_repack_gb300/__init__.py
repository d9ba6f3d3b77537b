"""Python binding of libw4a16.so, the GB300 W4A16 linear-layer library.

Argument marshalling only: every entry point below forwards device pointers,
sizes and the current CUDA stream to the C ABI declared in include/w4a16.h and
raises W4Error on a non-zero status. All computation runs in the library's CUDA
kernels; there is no fallback path. If the shared library has not been built
the first call raises, naming the build step.
"""
from __future__ import annotations

import contextlib
import ctypes
import os
from typing import Optional

import torch

__all__ = [
    "W4_F16", "W4_BF16", "W4_LAYOUT_STD", "W4_LAYOUT_TILE", "W4Error", "lib", "library_path",
    "dtype_code", "w4_status_string", "w4_last_cuda_error", "w4_abi_version", "w4_repack_sizes", "w4_repack_awq",
    "w4_repack_gptq", "w4a16_gemm_workspace_size", "w4a16_gemm", "w4a16_gemm_bias",
    "w4a16_gemm_noalloc", "w4a8_gemm_workspace_size", "w4a8_gemm", "linear_fp8",
    "w4_dequant", "gemm_workspace",
    "w4_device_status", "w4_test_stalled_gemm", "w4_test_prefill_plan",
    "RepackedLayer", "repack_awq", "repack_gptq", "linear", "w4a16_moe_gemm", "RepackedExperts",
    "repack_awq_experts", "moe_linear",
    "KV8Cache", "kv8_cache", "kv8_append", "kv8_attention", "w4_kv8_attention_workspace_size",
    "KV8Pool", "kv8_pool", "kv8_reserve", "kv8_fork", "kv8_free", "kv8_compact", "kv8_copy_pages",
    "w4_kv8_pages_workspace_size",
]

W4_F16, W4_BF16 = 0, 1
W4_LAYOUT_STD, W4_LAYOUT_TILE = 0, 1
W4_OK = 0
W4_ERR_CUDA = 9
W4_ERR_GIDX = 11

_PKG_DIR = os.path.dirname(os.path.abspath(__file__))
library_path = os.path.join(_PKG_DIR, "libw4a16.so")
_LIB: Optional[ctypes.CDLL] = None

_c_int, _c_size, _c_void_p = ctypes.c_int, ctypes.c_size_t, ctypes.c_void_p

class _KV8CacheStruct(ctypes.Structure):
    """w4_kv8_cache."""
    _fields_ = [("k", _c_void_p), ("v", _c_void_p), ("k_scale", _c_void_p),
                ("v_scale", _c_void_p), ("num_pages", _c_int), ("page_size", _c_int),
                ("kv_heads", _c_int), ("head_dim", _c_int)]


class _KV8HeadsStruct(ctypes.Structure):
    """w4_kv8_heads."""
    _fields_ = [("q_heads", _c_int), ("causal", _c_int), ("scale", ctypes.c_float)]


_SIGNATURES = {
    "w4_status_string": (ctypes.c_char_p, [_c_int]),
    "w4_last_cuda_error": (ctypes.c_char_p, []),
    "w4_abi_version": (_c_int, []),
    "w4_repack_sizes": (_c_int, [_c_int, _c_int, _c_int, _c_int, ctypes.POINTER(_c_size),
                                 ctypes.POINTER(_c_size), ctypes.POINTER(_c_size)]),
    "w4_repack_awq": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                               _c_int, _c_void_p, _c_void_p, _c_void_p, _c_void_p]),
    "w4_repack_gptq": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int, _c_int,
                                _c_int, _c_int, _c_int, _c_void_p, _c_void_p, _c_void_p,
                                _c_void_p, _c_void_p, _c_void_p]),
    "w4a16_gemm_workspace_size": (_c_size, [_c_int, _c_int, _c_int, _c_int, _c_int, _c_int]),
    "w4a16_gemm": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                            _c_int, _c_int, _c_int, _c_int, _c_int, _c_void_p, _c_size,
                            _c_void_p]),
    "w4a16_moe_gemm": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                _c_int, _c_int, _c_int, _c_int, _c_int, _c_int, _c_int,
                                _c_void_p]),
    "w4_test_stalled_gemm": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                      _c_int, _c_int, _c_int, _c_int, _c_int, _c_void_p]),
    "w4_test_prefill_plan": (_c_int, [_c_int, _c_int, _c_int, _c_int, ctypes.POINTER(_c_int)]),
    "w4a16_gemm_bias": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                 _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_int,
                                 _c_void_p, _c_size, _c_void_p]),
    "w4_dequant": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                            _c_int, _c_int, _c_void_p, _c_void_p]),
    "w4_device_status": (_c_int, [ctypes.POINTER(ctypes.c_int32), _c_int]),
    "w4a16_gemm_noalloc": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p,
                                    _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_int,
                                    _c_void_p]),
    "w4a8_gemm_workspace_size": (_c_size, [_c_int, _c_int]),
    "w4a8_gemm": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_void_p, _c_int,
                           _c_int, _c_int, _c_int, _c_int, _c_void_p, _c_size, _c_void_p]),
    "w4_kv8_append": (_c_int, [_c_void_p, _c_void_p, _c_size, _c_size, _c_void_p, _c_void_p, _c_int,
                               _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int, _c_void_p]),
    "w4_kv8_attention_workspace_size": (_c_size, [_c_int] * 7),
    "w4_kv8_attention": (_c_int, [_c_void_p, _c_size, _c_void_p, _c_void_p, _c_int, _c_void_p,
                                  _c_void_p, _c_void_p, _c_int, _c_int, _c_int, _c_int,
                                  _c_void_p, _c_int, _c_void_p, _c_size, _c_void_p]),
    "w4_kv8_pages_workspace_size": (_c_size, [_c_int, _c_int]),
    "w4_kv8_reserve": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_void_p, _c_int,
                                _c_void_p, _c_int, _c_void_p, _c_void_p, _c_size, _c_void_p]),
    "w4_kv8_fork": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_void_p, _c_int, _c_void_p,
                             _c_void_p, _c_int, _c_int, _c_void_p, _c_void_p, _c_void_p,
                             _c_void_p, _c_size, _c_void_p]),
    "w4_kv8_free": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_void_p, _c_int, _c_void_p,
                             _c_int, _c_int, _c_void_p, _c_void_p]),
    "w4_kv8_compact": (_c_int, [_c_void_p, _c_int, _c_void_p, _c_int, _c_int, _c_void_p,
                                _c_void_p, _c_void_p, _c_size, _c_void_p]),
    "w4_kv8_copy_pages": (_c_int, [_c_void_p, _c_void_p, _c_void_p, _c_int, _c_void_p]),
}


class W4Error(RuntimeError):
    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libw4a16.so (built in-tree); raise if it is missing."""
    global _LIB
    if _LIB is None:
        if not os.path.exists(library_path):
            raise RuntimeError(
                f"{library_path} is not built; run `python -c 'import __graft_entry__ as g; g.build()'`")
        L = ctypes.CDLL(library_path)
        for name, (res, args) in _SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _LIB = L
    return _LIB


def w4_status_string(status: int) -> str:
    return lib().w4_status_string(status).decode()


def w4_last_cuda_error() -> str:
    return lib().w4_last_cuda_error().decode()


def w4_abi_version() -> int:
    return lib().w4_abi_version()


def _check(status: int):
    if status != W4_OK:
        msg = w4_status_string(status)
        if status == W4_ERR_CUDA:
            msg += f" ({w4_last_cuda_error()})"
        raise W4Error(status, msg)


def _ptr(t) -> Optional[int]:
    if t is None:
        return None
    if isinstance(t, int):
        return t
    return t.data_ptr()


_RAW_STREAM = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream(stream, device_index: Optional[int] = None) -> Optional[int]:
    """The cudaStream_t handle to pass: `stream` itself (a torch stream or a raw
    handle), else torch's current stream on `device_index` (the current device
    when None)."""
    if stream is None:
        if not torch.cuda.is_available():
            return None
        if _RAW_STREAM is not None:
            if device_index is None:
                device_index = torch.cuda.current_device()
            return _RAW_STREAM(device_index)
        return torch.cuda.current_stream(device_index).cuda_stream
    if isinstance(stream, int):
        return stream
    return stream.cuda_stream


def dtype_code(dtype) -> int:
    if dtype in (W4_F16, W4_BF16):
        return dtype
    if dtype in (torch.float16, "fp16", "float16"):
        return W4_F16
    if dtype in (torch.bfloat16, "bf16", "bfloat16"):
        return W4_BF16
    raise ValueError(f"unsupported activation dtype {dtype}")


# --------------------------------------------------------------------------- #
# Raw entry points (same names and argument order as the C ABI)                 #
# --------------------------------------------------------------------------- #
def w4_repack_sizes(K: int, N: int, group: int, layout: int):
    a, b, c = _c_size(), _c_size(), _c_size()
    _check(lib().w4_repack_sizes(K, N, group, layout, ctypes.byref(a), ctypes.byref(b),
                                 ctypes.byref(c)))
    return a.value, b.value, c.value


def w4_repack_awq(qweight, qzeros, scales, K, N, group, dtype, layout, qw_out, zeros_out,
                  scales_out, stream=None):
    _check(lib().w4_repack_awq(_ptr(qweight), _ptr(qzeros), _ptr(scales), K, N, group,
                               dtype_code(dtype), layout, _ptr(qw_out), _ptr(zeros_out),
                               _ptr(scales_out), _stream(stream)))


def w4_repack_gptq(qweight, qzeros, scales, g_idx, K, N, group, dtype, layout, qw_out, zeros_out,
                   scales_out, perm_out=None, status_out=None, stream=None):
    _check(lib().w4_repack_gptq(_ptr(qweight), _ptr(qzeros), _ptr(scales), _ptr(g_idx), K, N,
                                group, dtype_code(dtype), layout, _ptr(qw_out), _ptr(zeros_out),
                                _ptr(scales_out), _ptr(perm_out), _ptr(status_out),
                                _stream(stream)))


def w4a16_gemm_workspace_size(M, N, K, group, dtype, has_perm) -> int:
    return lib().w4a16_gemm_workspace_size(M, N, K, group, dtype_code(dtype), int(bool(has_perm)))


def w4a16_gemm(x, qw, scales, zeros, perm, y, M, N, K, group, dtype, workspace=None,
               workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().w4a16_gemm(_ptr(x), _ptr(qw), _ptr(scales), _ptr(zeros), _ptr(perm), _ptr(y),
                            M, N, K, group, dtype_code(dtype), _ptr(workspace), workspace_bytes,
                            _stream(stream)))


def w4a16_gemm_bias(x, qw, scales, zeros, perm, bias, y, M, N, K, group, dtype, workspace=None,
                    workspace_bytes=None, stream=None):
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().w4a16_gemm_bias(_ptr(x), _ptr(qw), _ptr(scales), _ptr(zeros), _ptr(perm),
                                 _ptr(bias), _ptr(y), M, N, K, group, dtype_code(dtype),
                                 _ptr(workspace), workspace_bytes, _stream(stream)))


def w4a16_moe_gemm(x, qw, scales, zeros, expert_offsets, y, num_experts, max_rows_per_expert,
                   total_rows, N, K, group, dtype, stream=None):
    _check(lib().w4a16_moe_gemm(_ptr(x), _ptr(qw), _ptr(scales), _ptr(zeros), _ptr(expert_offsets),
                                _ptr(y), num_experts, max_rows_per_expert, total_rows, N, K, group,
                                dtype_code(dtype), _stream(stream)))


class RepackedExperts:
    """Device buffers of an MoE layer's experts, one expert after another."""

    def __init__(self, E, K, N, group, dtype, qw, zeros, scales):
        self.E, self.K, self.N, self.group, self.dtype = E, K, N, group, dtype
        self.qw, self.zeros, self.scales = qw, zeros, scales


def repack_awq_experts(qweights, qzeros, scales, K, N, group, dtype, stream=None):
    """Per-expert w4_repack_awq (TILE layout) into stacked buffers: qweights /
    qzeros / scales are sequences of the experts' checkpoint tensors (qzeros
    entries may be None for symmetric experts)."""
    E = len(qweights)
    qw_b, z_b, s_b = w4_repack_sizes(K, N, group, W4_LAYOUT_TILE)
    dev = qweights[0].device
    qw = torch.empty(E * qw_b // 4, dtype=torch.int32, device=dev)
    zeros = torch.empty(E * z_b // 4, dtype=torch.int32, device=dev)
    sc = torch.empty(E * s_b // 2, dtype=_half_dtype(dtype), device=dev)
    nq, nz, ns = qw_b // 4, z_b // 4, s_b // 2
    for e in range(E):
        w4_repack_awq(qweights[e], qzeros[e], scales[e], K, N, group, dtype, W4_LAYOUT_TILE,
                      qw[e * nq:(e + 1) * nq], zeros[e * nz:(e + 1) * nz],
                      sc[e * ns:(e + 1) * ns], stream)
    return RepackedExperts(E, K, N, group, dtype, qw, zeros, sc)


def moe_linear(x, experts: RepackedExperts, expert_offsets, max_rows_per_expert, y=None,
               stream=None):
    """y[m] = x[m] · W_e for the rows m of expert e ([off[e], off[e+1]), x sorted
    by expert); expert_offsets: int32 [E + 1] on the device."""
    T = x.shape[0]
    if y is None:
        y = torch.empty((T, experts.N), dtype=x.dtype, device=x.device)
    w4a16_moe_gemm(x, experts.qw, experts.scales, experts.zeros, expert_offsets, y, experts.E,
                   max_rows_per_expert, T, experts.N, experts.K, experts.group, experts.dtype,
                   stream)
    return y


def w4_test_stalled_gemm(x, qw, scales, zeros, y, M, N, K, group, dtype, stream=None):
    """The small-M GEMM with its weight copies withheld (the timeout test hook)."""
    _check(lib().w4_test_stalled_gemm(_ptr(x), _ptr(qw), _ptr(scales), _ptr(zeros), _ptr(y), M, N,
                                      K, group, dtype_code(dtype), _stream(stream)))


def w4_test_prefill_plan(M, N, K, sm_count):
    """The large-M kernel's plan for an M x N x K call on sm_count SMs (host
    only): (rows per tile, output tiles, split tiles, K slices of each)."""
    out = (_c_int * 4)()
    _check(lib().w4_test_prefill_plan(M, N, K, sm_count, out))
    return tuple(out)


def w4a16_gemm_noalloc(x, qw, scales, zeros, perm, y, M, N, K, group, dtype, stream=None):
    """w4a16_gemm for callers that cannot allocate device memory: act-order
    staging goes to the library's static device array instead of a workspace."""
    _check(lib().w4a16_gemm_noalloc(_ptr(x), _ptr(qw), _ptr(scales), _ptr(zeros), _ptr(perm),
                                    _ptr(y), M, N, K, group, dtype_code(dtype), _stream(stream)))


def w4a8_gemm_workspace_size(M, K) -> int:
    return lib().w4a8_gemm_workspace_size(M, K)


def w4a8_gemm(x, qw, scales, zeros, y, M, N, K, group, dtype, workspace, workspace_bytes=None,
              stream=None):
    """INT4 weights x per-tensor FP8 activations (quantised on the device)."""
    if workspace_bytes is None:
        workspace_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().w4a8_gemm(_ptr(x), _ptr(qw), _ptr(scales), _ptr(zeros), _ptr(y), M, N, K, group,
                           dtype_code(dtype), _ptr(workspace), workspace_bytes, _stream(stream)))


def w4_device_status(clear: bool = False) -> int:
    v = ctypes.c_int32(0)
    _check(lib().w4_device_status(ctypes.byref(v), int(bool(clear))))
    return v.value


def w4_dequant(qw, scales, zeros, K, N, group, dtype, layout, out_f32, w_out, stream=None):
    _check(lib().w4_dequant(_ptr(qw), _ptr(scales), _ptr(zeros), K, N, group, dtype_code(dtype),
                            layout, int(bool(out_f32)), _ptr(w_out), _stream(stream)))


# --------------------------------------------------------------------------- #
# Convenience: allocate outputs with torch, then call the entry points          #
# --------------------------------------------------------------------------- #
class RepackedLayer:
    """Device buffers of one repacked layer (what the GEMM reads)."""

    def __init__(self, K, N, group, dtype, layout, qw, zeros, scales, perm=None, status=None):
        self.K, self.N, self.group, self.dtype, self.layout = K, N, group, dtype, layout
        self.qw, self.zeros, self.scales, self.perm, self.status = qw, zeros, scales, perm, status


def _half_dtype(dtype) -> torch.dtype:
    return torch.bfloat16 if dtype_code(dtype) == W4_BF16 else torch.float16


def _alloc_repacked(K, N, group, dtype, layout, device):
    qw_b, z_b, s_b = w4_repack_sizes(K, N, group, layout)
    qw = torch.empty(qw_b // 4, dtype=torch.int32, device=device)
    zeros = torch.empty(z_b // 4, dtype=torch.int32, device=device)
    scales = torch.empty(s_b // 2, dtype=_half_dtype(dtype), device=device)
    return qw, zeros, scales


def repack_awq(qweight, qzeros, scales, K, N, group, dtype, layout=W4_LAYOUT_TILE, stream=None):
    qw, zeros, sc = _alloc_repacked(K, N, group, dtype, layout, qweight.device)
    w4_repack_awq(qweight, qzeros, scales, K, N, group, dtype, layout, qw, zeros, sc, stream)
    return RepackedLayer(K, N, group, dtype, layout, qw, zeros, sc)


def repack_gptq(qweight, qzeros, scales, g_idx, K, N, group, dtype, layout=W4_LAYOUT_TILE,
                stream=None):
    qw, zeros, sc = _alloc_repacked(K, N, group, dtype, layout, qweight.device)
    perm = status = None
    if g_idx is not None:
        perm = torch.empty(K, dtype=torch.int32, device=qweight.device)
        status = torch.full((4,), -1, dtype=torch.int32, device=qweight.device)
    w4_repack_gptq(qweight, qzeros, scales, g_idx, K, N, group, dtype, layout, qw, zeros, sc,
                   perm, status, stream)
    return RepackedLayer(K, N, group, dtype, layout, qw, zeros, sc, perm, status)


_WORKSPACES: dict = {}  # (device, stream) -> every block handed out, the largest last


def _on_stream(stream, idx):
    """A context in which torch works on `stream` of device idx (None: the current one)."""
    if stream is None:
        return contextlib.nullcontext()
    if isinstance(stream, int):
        stream = (torch.cuda.ExternalStream(stream, device=torch.device("cuda", idx)) if stream
                  else torch.cuda.default_stream(idx))
    return torch.cuda.stream(stream)


def gemm_workspace(nbytes: int, device, stream=None):
    """A workspace of at least nbytes on `device` for calls on `stream`, kept
    and reused across calls (calls on one stream run in order, so they can
    share it, and no call allocates device memory once it is big enough). A
    block that a larger one replaces is kept too, for as long as the process
    runs: a captured graph goes on using its address. Blocks grow by half at
    least, so those kept are at most twice the last one."""
    dev = torch.device(device)
    idx = dev.index if dev.index is not None else torch.cuda.current_device()
    handle = _stream(stream, idx)
    key = (idx, handle)
    blocks = _WORKSPACES.setdefault(key, [])
    if not blocks or blocks[-1].numel() < nbytes:
        least = blocks[-1].numel() * 3 // 2 if blocks else 256
        with _on_stream(stream, idx):
            blocks.append(torch.empty(max(nbytes, least), dtype=torch.uint8, device=dev))
    return blocks[-1]


_WS_SIZES: dict = {}
_WS_SIZES_MAX = 4096


def _workspace_size_cached(M, layer: RepackedLayer, device) -> int:
    """w4a16_gemm_workspace_size for (device, M, layer shape), remembered: the
    size depends only on those (and on the device's SM count), and linear()
    would otherwise pay a second library call on every call."""
    dev = device.index if device.index is not None else -1
    key = (dev, M, layer.N, layer.K, layer.group, layer.dtype, layer.perm is not None)
    need = _WS_SIZES.get(key)
    if need is None:
        need = w4a16_gemm_workspace_size(M, layer.N, layer.K, layer.group, layer.dtype,
                                         layer.perm is not None)
        if len(_WS_SIZES) >= _WS_SIZES_MAX:
            _WS_SIZES.clear()
        _WS_SIZES[key] = need
    return need


def linear_fp8(x, layer: RepackedLayer, y=None, workspace=None, stream=None):
    """y = x · W with the activations quantised per tensor to e4m3 on the device
    and the product on the fp8 tensor cores (w4a8_gemm); layer without act-order,
    group 128 or -1."""
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, layer.N), dtype=x.dtype, device=x.device)
    if M == 0:
        return y
    if workspace is None:
        workspace = gemm_workspace(w4a8_gemm_workspace_size(M, layer.K), x.device, stream)
    w4a8_gemm(x, layer.qw, layer.scales, layer.zeros, y, M, layer.N, layer.K, layer.group,
              layer.dtype, workspace, None, stream)
    return y


def linear(x, layer: RepackedLayer, y=None, workspace=None, stream=None, bias=None):
    """y = x · W (+ bias) for a TILE-layout layer; x is [M, K] fp16/bf16 on the
    device, bias [N] in the same dtype or None. Without `workspace`, the one kept
    for (device, stream) is used (grown as needed)."""
    M = x.shape[0]
    if y is None:
        y = torch.empty((M, layer.N), dtype=x.dtype, device=x.device)
    need = _workspace_size_cached(M, layer, x.device)
    if need and workspace is None:
        workspace = gemm_workspace(need, x.device, stream)
    handle = _stream(stream, x.device.index)
    ws_bytes = 0 if workspace is None else workspace.numel() * workspace.element_size()
    _check(lib().w4a16_gemm_bias(x.data_ptr(), layer.qw.data_ptr(), layer.scales.data_ptr(),
                                 layer.zeros.data_ptr(), _ptr(layer.perm), _ptr(bias),
                                 y.data_ptr(), M, layer.N, layer.K, layer.group,
                                 dtype_code(layer.dtype), _ptr(workspace), ws_bytes, handle))
    return y


# --------------------------------------------------------------------------- #
# 8-bit key-value cache                                                         #
# --------------------------------------------------------------------------- #
# A decode step makes these calls once a layer with a few microseconds of work
# each, so the wrappers look at every tensor once and keep what does not change.
_F8, _F32, _I32 = torch.float8_e4m3fn, torch.float32, torch.int32
_HALF_CODES = {torch.float16: W4_F16, torch.bfloat16: W4_BF16}


class _Handle:
    """Keeps the addresses of its tensors, so its attributes cannot be set anew."""

    def __setattr__(self, name, value):
        if name in self.__dict__ and not name.startswith("_"):
            raise AttributeError(f"{type(self).__name__}.{name} cannot be set: make a new {type(self).__name__}")
        self.__dict__[name] = value


class KV8Cache(_Handle):
    """One layer's cache: k and v float8_e4m3fn [pages, kv_heads, page, head_dim],
    k_scale and v_scale float32 [pages, kv_heads], all contiguous on the GPU."""

    def __init__(self, k, v, k_scale, v_scale):
        if k.dim() != 4 or v.shape != k.shape or k.dtype is not _F8 or v.dtype is not _F8:
            raise ValueError("k and v must be float8_e4m3fn [pages, kv_heads, page, head_dim]")
        if k_scale.shape != k.shape[:2] or v_scale.shape != k.shape[:2] or \
                k_scale.dtype is not _F32 or v_scale.dtype is not _F32:
            raise ValueError("k_scale and v_scale must be float32 [pages, kv_heads]")
        if not (k.is_contiguous() and v.is_contiguous() and k_scale.is_contiguous()
                and v_scale.is_contiguous()):
            raise ValueError("the cache's tensors must be contiguous")
        if not k.device == v.device == k_scale.device == v_scale.device:
            raise ValueError("the cache's tensors must be on one device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.num_pages, self.kv_heads, self.page_size, self.head_dim = k.shape
        self._struct = _KV8CacheStruct(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(),
                                       v_scale.data_ptr(), self.num_pages, self.page_size,
                                       self.kv_heads, self.head_dim)
        self._ref = ctypes.addressof(self._struct)
        self._device = k.get_device()


def kv8_cache(num_pages, kv_heads, page_size, head_dim, device="cuda") -> KV8Cache:
    """An empty cache."""
    shape = (num_pages, kv_heads, page_size, head_dim)
    k, v = (torch.zeros(shape, dtype=torch.uint8, device=device).view(_F8) for _ in range(2))
    ks, vs = (torch.ones(shape[:2], dtype=_F32, device=device) for _ in range(2))
    return KV8Cache(k, v, ks, vs)


_CURRENT_DEVICE = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _one_gpu(index, *tensors):
    """Refuses tensors that are not on GPU `index`, and a GPU that is not the current
    one: the kernels would take their addresses for its own."""
    for x in tensors:
        if x.get_device() != index:
            raise ValueError("all tensors of a call must be on the same GPU")
    if index < 0:
        raise ValueError("the tensors must be on a GPU")
    if _CURRENT_DEVICE() != index:
        raise ValueError(f"the tensors are on GPU {index}, which is not the current one")


def _on(stream, index):
    """The stream handle for tensors on device `index` (-1: not on a GPU)."""
    if stream is None and index >= 0 and _RAW_STREAM is not None:
        return _RAW_STREAM(index)
    return _stream(stream, index if index >= 0 else None)


def _new(make, stream, index):
    """make()'s tensor for a call on `stream`: allocated there, so that nothing that still
    runs on the current stream uses its memory, and kept for both when it is let go."""
    if stream is None:
        return make()
    with _on_stream(stream, index):
        x = make()
    x.record_stream(torch.cuda.current_stream(index))
    return x


def _rows(x, name, heads, dim):
    """The token stride of x [tokens, heads, dim], whose rows may be slices of a
    wider buffer but whose heads and elements are adjacent."""
    shape = x.shape
    if len(shape) != 3 or shape[1] != heads or shape[2] != dim:
        raise ValueError(f"{name} must be [tokens, {heads}, {dim}], not {tuple(shape)}")
    st = x.stride()
    if shape[0] and (st[2] != 1 or (st[1] != dim and heads > 1)):
        raise ValueError(f"{name}: heads and elements of a token must be adjacent in memory")
    return st[0] if shape[0] > 1 else heads * dim


def _ints(x, name):
    """The address of a contiguous int32 array."""
    if x.dtype is not _I32 or not x.is_contiguous():
        raise ValueError(f"{name} must be contiguous int32")
    return x.data_ptr()


def _table(x, stream, index):
    """(address, pages of a row, tensor to hold on to) of a table [sequences, pages].
    The kernels take a row's stride for its length, so columns of a wider table are
    copied, on the call's stream."""
    if x.dim() != 2 or x.dtype is not _I32:
        raise ValueError("the table must be int32 [sequences, pages]")
    if not x.is_contiguous():
        with _on_stream(stream if index >= 0 else None, index):
            x = x.contiguous()
    return x.data_ptr(), x.shape[1], x


def _batch(table, kv_lens, cu_q):
    b = kv_lens.shape[0]
    if table.shape[0] < b or cu_q.shape[0] != b + 1:
        raise ValueError("table needs a row and cu_q a bound for every entry of kv_lens")
    return b


def kv8_append(k, v, cache: KV8Cache, table, kv_lens, cu_q, max_q_len, stream=None):
    """Quantises new keys and values k, v [tokens, kv_heads, head_dim] (fp16 or
    bf16, packed by sequence: rows cu_q[b] .. cu_q[b + 1]) into the cache as each
    sequence's last tokens: kv_lens [batch] counts them already. table [batch,
    pages] int32 gives the sequences' pages. See w4_kv8_append in include/w4a16.h."""
    dtype = k.dtype
    if v.dtype is not dtype or v.shape != k.shape:
        raise ValueError("k and v must have the same type and shape")
    hk, d = cache.kv_heads, cache.head_dim
    code = _HALF_CODES.get(dtype)
    if code is None:
        code = dtype_code(dtype)
    _one_gpu(cache._device, k, v, table, kv_lens, cu_q)
    tab, stride, held = _table(table, stream, cache._device)
    status = lib().w4_kv8_append(
        k.data_ptr(), v.data_ptr(), _rows(k, "k", hk, d), _rows(v, "v", hk, d), cache._ref, tab,
        stride, _ints(kv_lens, "kv_lens"), _ints(cu_q, "cu_q"), _batch(table, kv_lens, cu_q),
        k.shape[0], max_q_len, code, _on(stream, cache._device))
    if status:
        _check(status)


def w4_kv8_attention_workspace_size(batch, total_q, max_q_len, max_kv_len, q_heads, kv_heads,
                                    head_dim) -> int:
    return lib().w4_kv8_attention_workspace_size(batch, total_q, max_q_len, max_kv_len, q_heads,
                                                 kv_heads, head_dim)


_KV8_HEADS: dict = {}   # (q_heads, causal, scale) -> (struct, address)
_KV8_SIZES: dict = {}   # arguments of a workspace size -> bytes
_KV8_SPACES: dict = {}  # (device, stream) -> (address, bytes) of a block of gemm_workspace
_KV8_KEPT = 4096


def _keep(kept, key, value):
    if len(kept) >= _KV8_KEPT:
        kept.clear()
    kept[key] = value
    return value


def _space(nbytes, index, handle, stream):
    """(address, bytes) of gemm_workspace's block for a device and stream."""
    got = _KV8_SPACES.get((index, handle))
    if got is None or got[1] < nbytes:
        t = gemm_workspace(nbytes, torch.device("cuda", index), stream)
        got = _keep(_KV8_SPACES, (index, handle), (t.data_ptr(), t.numel()))
    return got


def kv8_attention(q, cache: KV8Cache, table, kv_lens, cu_q, max_q_len, max_kv_len, scale=None,
                  causal=True, out=None, workspace=None, stream=None):
    """Attention of q [tokens, q_heads, head_dim] (fp16 or bf16, packed by
    sequence as for kv8_append) over each sequence's kv_lens[b] cached tokens;
    causal: its queries are its last tokens; otherwise each sees all of them.
    scale defaults to head_dim ** -0.5. Without `workspace`, the one kept for
    (device, stream) is used. See w4_kv8_attention in include/w4a16.h."""
    shape, dtype, dim = q.shape, q.dtype, cache.head_dim
    tokens, heads = shape[0], shape[1]
    stride = _rows(q, "q", heads, dim)
    batch = _batch(table, kv_lens, cu_q)
    if heads % cache.kv_heads:
        raise W4Error(2, w4_status_string(2))
    code = _HALF_CODES.get(dtype)
    if code is None:
        code = dtype_code(dtype)
    if out is not None and (out.shape != shape or out.dtype is not dtype or not out.is_contiguous()):
        raise ValueError("out must be contiguous, with q's shape and type")
    index = cache._device
    _one_gpu(index, q, q if out is None else out, table, kv_lens, cu_q)
    if out is None:
        out = _new(lambda: torch.empty_like(q, memory_format=torch.contiguous_format), stream, index)
    how = _KV8_HEADS.get((heads, causal, scale))
    if how is None:
        struct = _KV8HeadsStruct(heads, causal, dim ** -0.5 if scale is None else scale)
        how = (struct, ctypes.addressof(struct))
        if scale is not None:
            _keep(_KV8_HEADS, (heads, causal, scale), how)
    L = lib()
    key = (batch, tokens, max_q_len, max_kv_len, heads, cache.kv_heads, dim)
    nbytes = _KV8_SIZES.get(key)
    if nbytes is None:
        nbytes = _keep(_KV8_SIZES, key, L.w4_kv8_attention_workspace_size(*key))
    handle = _on(stream, index)
    space = None
    if workspace is not None:
        _one_gpu(index, workspace)
        if not workspace.is_contiguous():
            raise ValueError("the workspace must be contiguous")
        space, nbytes = workspace.data_ptr(), workspace.numel() * workspace.element_size()
    elif nbytes:
        space, nbytes = _space(nbytes, index, handle, stream)
    tab, tab_stride, held = _table(table, stream, index)
    status = L.w4_kv8_attention(
        q.data_ptr(), stride, cache._ref, tab, tab_stride, _ints(kv_lens, "kv_lens"),
        _ints(cu_q, "cu_q"), out.data_ptr(), batch, tokens, max_q_len, max_kv_len, how[1], code,
        space, nbytes, handle)
    if status:
        _check(status)
    return out


class KV8Pool(_Handle):
    """The pages of a pool and the sequences that hold them: refs [pages] (0: a
    free page), table [sequences, pages of the longest] (-1 past a sequence's
    pages), lens [sequences] (tokens; 0: an empty slot), int32 on the GPU.
    status: an int32 tensor that receives each call's W4_OK or error (a call
    that fails changes nothing, but kv8_free ends the sequences that it can);
    without one, errors go to w4_device_status.
    The three are changed in place, and table's row is a sequence's whole list of
    pages: columns of a wider table are refused."""

    def __init__(self, refs, table, lens, page_size, status=None):
        pages, seqs = refs.shape[0], lens.shape[0]
        if table.dim() != 2 or table.shape[0] != seqs:
            raise ValueError("table must be [sequences, pages], lens [sequences]")
        if not refs.device == table.device == lens.device or \
                (status is not None and status.device != refs.device):
            raise ValueError("the pool's tensors must be on one device")
        # what any of the calls needs: at most a pair or a sequence for every slot
        nbytes = _KV8_SIZES.get((pages, seqs))
        if nbytes is None:
            nbytes = _keep(_KV8_SIZES, (pages, seqs), w4_kv8_pages_workspace_size(pages, seqs))
        self.__dict__.update(  # (a program may make one for every step)
            refs=refs, table=table, lens=lens, page_size=page_size, status=status,
            _args=(_ints(refs, "refs"), pages, _ints(table, "table"), table.shape[1],
                   _ints(lens, "lens"), seqs),
            _status=None if status is None else _ints(status, "status"),
            _device=refs.get_device(), _bytes=nbytes)


def kv8_pool(num_pages, num_seqs, max_len, page_size, device="cuda") -> KV8Pool:
    """A pool of free pages with num_seqs empty sequences of at most max_len tokens."""
    return KV8Pool(torch.zeros(num_pages, dtype=_I32, device=device),
                   torch.full((num_seqs, -(-max_len // page_size)), -1, dtype=_I32, device=device),
                   torch.zeros(num_seqs, dtype=_I32, device=device), page_size,
                   torch.zeros(1, dtype=_I32, device=device))


def w4_kv8_pages_workspace_size(num_pages, n) -> int:
    return lib().w4_kv8_pages_workspace_size(num_pages, n)


def kv8_reserve(pool: KV8Pool, new_tokens, stream=None):
    """Lengthens every sequence s by new_tokens[s] and gives it the pages that
    takes, the lowest free ones in order."""
    if new_tokens.shape[0] != pool._args[5]:
        raise ValueError("new_tokens must have an entry for every sequence")
    _one_gpu(pool._device, new_tokens)
    handle = _on(stream, pool._device)
    status = lib().w4_kv8_reserve(*pool._args, _ints(new_tokens, "new_tokens"), pool.page_size,
                                  pool._status,
                                  *_space(pool._bytes, pool._device, handle, stream), handle)
    if status:
        _check(status)


def kv8_fork(pool: KV8Pool, src, dst, stream=None):
    """Makes each empty sequence dst[i] a copy of src[i] that shares its full
    pages. Returns (copy_src, copy_dst): the last partial pages to copy with
    kv8_copy_pages in every layer's cache (-1 where there is none)."""
    n = src.shape[0]
    if dst.shape[0] != n:
        raise ValueError("src and dst must have the same length")
    _one_gpu(pool._device, src, dst)
    copy_src, copy_dst = _new(lambda: torch.empty((2, n), dtype=_I32, device=src.device), stream,
                              pool._device).unbind()
    handle = _on(stream, pool._device)
    status = lib().w4_kv8_fork(*pool._args, _ints(src, "src"), _ints(dst, "dst"), n,
                               pool.page_size, copy_src.data_ptr(), copy_dst.data_ptr(),
                               pool._status, *_space(pool._bytes, pool._device, handle, stream),
                               handle)
    if status:
        _check(status)
    return copy_src, copy_dst


def kv8_free(pool: KV8Pool, seqs, stream=None):
    """Ends the sequences: their pages lose a reference, their slots become empty."""
    _one_gpu(pool._device, seqs)
    status = lib().w4_kv8_free(*pool._args, _ints(seqs, "seqs"), seqs.shape[0], pool.page_size,
                               pool._status, _on(stream, pool._device))
    if status:
        _check(status)


def kv8_compact(pool: KV8Pool, stream=None):
    """Renumbers the pages in use to the front of the pool. Returns (copy_src,
    copy_dst) for kv8_copy_pages in every layer's cache (-1 after the last)."""
    _one_gpu(pool._device)
    refs, pages, tab, stride, _, seqs = pool._args
    copy_src, copy_dst = _new(lambda: torch.empty((2, pages), dtype=_I32, device=pool.refs.device),
                              stream, pool._device).unbind()
    handle = _on(stream, pool._device)
    status = lib().w4_kv8_compact(refs, pages, tab, stride, seqs, copy_src.data_ptr(),
                                  copy_dst.data_ptr(),
                                  *_space(pool._bytes, pool._device, handle, stream), handle)
    if status:
        _check(status)
    return copy_src, copy_dst


def kv8_copy_pages(cache: KV8Cache, src, dst, stream=None):
    """Copies page src[i] to page dst[i], codes and scales (entries below 0: none)."""
    n = src.shape[0]
    if dst.shape[0] != n:
        raise ValueError("src and dst must have the same length")
    _one_gpu(cache._device, src, dst)
    status = lib().w4_kv8_copy_pages(cache._ref, _ints(src, "src"), _ints(dst, "dst"), n,
                                     _on(stream, cache._device))
    if status:
        _check(status)
