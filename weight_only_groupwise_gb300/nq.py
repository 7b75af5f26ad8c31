"""Thin ctypes binding of libnq.so (include/nq.h). Argument marshalling only: every step of
the projection runs in the library's CUDA kernels. PyTorch provides device memory and the
current stream. There is no fallback: if the library is missing or the device is not a GB300
(sm_103), the calls raise.

`stream`: where a call runs (None: the current stream). The caller orders it behind what writes the call's
inputs, and what reads the results behind it. Results that a call makes itself are memory of that stream.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libnq.so")
_lib = None

STATUS = {0: "NQ_OK", -1: "NQ_ERR_NULL", -2: "NQ_ERR_SHAPE", -3: "NQ_ERR_ALIGN", -4: "NQ_ERR_ALIAS",
          -5: "NQ_ERR_CUDA", -6: "NQ_ERR_DEVICE", -7: "NQ_ERR_TIMEOUT", -8: "NQ_ERR_SCRATCH"}


class NqGroup(ctypes.Structure):
    """struct nq_group of include/nq.h."""
    _fields_ = [("Wq", ctypes.c_void_p), ("S", ctypes.c_void_p), ("Y", ctypes.c_void_p), ("N", ctypes.c_int)]


class NqError(RuntimeError):
    def __init__(self, status: int, msg: str):
        super().__init__(msg)
        self.status = status


def lib() -> ctypes.CDLL:
    """Load libnq.so (built by weight_only_groupwise_gb300.build). Raises if it is missing."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(f"{LIB_PATH} is missing: run weight_only_groupwise_gb300.build.build() "
                               "(the CUDA library is required; there is no CPU path)")
        L = ctypes.CDLL(LIB_PATH)
        P, I, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t
        L.nq_status_string.argtypes = [I]
        L.nq_status_string.restype = ctypes.c_char_p
        L.nq_version.restype = I
        for f in ("nq_packed_bytes_q4", "nq_packed_bytes_q5"):
            getattr(L, f).argtypes = [I, I]
            getattr(L, f).restype = S
        L.nq_scale_bytes.argtypes = [I, I]
        L.nq_scale_bytes.restype = S
        L.nq_pack_q4.argtypes = [P, P, I, I, P, P, P]
        L.nq_pack_q5.argtypes = [P, P, P, I, I, P, P, P]
        L.nq_gemm_q4.argtypes = [P, P, P, P, I, I, I, P]
        L.nq_gemm_q5.argtypes = [P, P, P, P, I, I, I, P]
        L.nq_gemm_q4_noalloc.argtypes = [P, P, P, P, I, I, I, P]
        L.nq_swiglu_q4.argtypes = [P, P, P, P, P, P, I, I, I, P]
        L.nq_swiglu_q5.argtypes = [P, P, P, P, P, P, I, I, I, P]
        for f in ("nq_dequant_q4_debug", "nq_dequant_q5_debug", "nq_dequant_q4_debug_bf16",
                  "nq_dequant_q5_debug_bf16"):
            getattr(L, f).argtypes = [P, P, P, I, I, P]
            getattr(L, f).restype = I
        L.nq_packed_bytes_fp4.argtypes = [I, I]
        L.nq_packed_bytes_fp4.restype = S
        L.nq_scale_bytes_fp4.argtypes = [I, I]
        L.nq_scale_bytes_fp4.restype = S
        L.nq_pack_fp4.argtypes = [P, P, I, I, P, P, P]
        L.nq_pack_fp4.restype = I
        L.nq_gemm_fp4.argtypes = [P, P, P, ctypes.c_float, P, I, I, I, P]
        L.nq_gemm_fp4.restype = I
        L.nq_swiglu_fp4.argtypes = [P, P, P, ctypes.c_float, P, P, ctypes.c_float, P, I, I, I, P]
        L.nq_swiglu_fp4.restype = I
        L.nq_dequant_fp4_debug.argtypes = [P, P, ctypes.c_float, P, I, I, P]
        L.nq_dequant_fp4_debug.restype = I
        for f in ("nq_gemm_q4_grouped", "nq_gemm_q5_grouped"):
            getattr(L, f).argtypes = [P, P, I, I, I, P]
            getattr(L, f).restype = I
        L.nq_reserve.argtypes = [I, I, I]
        L.nq_device_error.argtypes = []
        L.nq_wait_limit.argtypes = [ctypes.c_longlong]
        L.nq_wait_limit.restype = ctypes.c_longlong
        L.nq_shutdown.argtypes = []
        L.nq_shutdown.restype = None
        L.nq_plan_info.argtypes = [I, I, I, I, I, I, P]
        L.nq_plan_segments.argtypes = [I, I, I, I, I, I, I, P, ctypes.c_int64]
        L.nq_plan_segments.restype = ctypes.c_int64
        L.nq_tensor_core_batches.argtypes = [I]
        L.nq_tensor_core_batches.restype = I
        L.nq_plan_tc_info.argtypes = [I, I, I, I, I, P]
        L.nq_plan_tc_info.restype = I
        L.nq_route_info.argtypes = [I, I, I, I, I, I, P]
        L.nq_route_info.restype = I
        L.nq_slab_clusters.argtypes = [I]
        L.nq_slab_clusters.restype = I
        L.nq_plan_cluster_info.argtypes = [I, I, I, I, I, I, P]
        L.nq_plan_cluster_segments.argtypes = [I, I, I, I, I, I, I, P, ctypes.c_int64]
        L.nq_plan_cluster_segments.restype = ctypes.c_int64
        L.nq_program_create.argtypes = [ctypes.POINTER(ctypes.c_void_p)]
        L.nq_program_gemm.argtypes = [P, I, P, P, P, P, I, I, I]
        L.nq_program_gemm_fp4.argtypes = [P, P, P, P, ctypes.c_float, P, I, I, I]
        L.nq_program_swiglu.argtypes = [P, I, P, P, P, P, P, P, I, I, I]
        L.nq_program_grouped.argtypes = [P, I, P, P, I, I, I]
        L.nq_program_swiglu_fp4.argtypes = [P, P, P, P, ctypes.c_float, P, P, ctypes.c_float, P, I, I, I]
        L.nq_program_build.argtypes = [P]
        L.nq_program_launch.argtypes = [P, P]
        L.nq_program_info.argtypes = [P, P]
        for f in ("nq_program_create", "nq_program_gemm", "nq_program_gemm_fp4", "nq_program_swiglu", "nq_program_swiglu_fp4",
                  "nq_program_grouped", "nq_program_build", "nq_program_launch", "nq_program_info"):
            getattr(L, f).restype = I
        L.nq_program_destroy.argtypes = [P]
        L.nq_program_destroy.restype = None
        LL, F = ctypes.c_longlong, ctypes.c_float
        L.nq_page_tables.argtypes = [P, P, I, P, I, P, I, P, LL, I, P, P, P, P, I, P, P]
        L.nq_kv_append.argtypes = [P, LL, P, LL, P, I, P, P]
        L.nq_attn_paged.argtypes = [P, LL, P, P, LL, I, P, P, I, I, I, F, I, I, I, P, LL, P]
        L.nq_attn_reserve.argtypes = []
        L.nq_sample.argtypes = [P, I, LL, P, LL, I, I, P, P, P, P, P, P]
        L.nq_quant_fp8.argtypes = [P, I, LL, I, I, P, LL, P, LL, P]
        L.nq_gemm_fp8.argtypes = [P, P, P, I, I, P]
        L.nq_swiglu_fp8.argtypes = [P, P, P, P, I, I, P]
        L.nq_gemm_fp8_experts.argtypes = [P, P, I, P, I, P, P, I, I, P, P]
        L.nq_swiglu_fp8_experts.argtypes = [P, P, I, P, I, P, P, P, I, I, P, P]
        L.nq_fp8_scratch_bytes.argtypes = [I, I, I, I]
        L.nq_fp8_scratch_bytes.restype = S
        L.nq_moe_route.argtypes = [P, I, LL, P, I, I, I, I, I, F, P, P, P, P, P, P]
        L.nq_moe_combine.argtypes = [P, I, LL, I, P, P, I, I, I, P, LL, P, LL, P]
        for f in ("nq_quant_fp8", "nq_gemm_fp8", "nq_swiglu_fp8", "nq_gemm_fp8_experts", "nq_swiglu_fp8_experts",
                  "nq_moe_route", "nq_moe_combine"):
            getattr(L, f).restype = I
        for f in ("nq_sample", "nq_page_tables", "nq_kv_append", "nq_attn_paged", "nq_attn_reserve"):
            getattr(L, f).restype = I
        for f in ("nq_pack_q4", "nq_pack_q5", "nq_gemm_q4", "nq_gemm_q5", "nq_gemm_q4_noalloc", "nq_swiglu_q4",
                  "nq_swiglu_q5", "nq_reserve", "nq_device_error", "nq_plan_info", "nq_plan_cluster_info"):
            getattr(L, f).restype = I
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().nq_status_string(int(status)).decode()


def _check(status: int) -> None:
    if status != 0:
        raise NqError(status, status_string(status))


def _ptr(t):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream):
    if stream is None:
        stream = torch.cuda.current_stream()
    return ctypes.c_void_p(stream.cuda_stream)


def _own(stream):
    """A context in which tensors are made for kernels on `stream`, of its own memory: the current stream's free memory may
    still be written by what waits there."""
    return torch.cuda.stream(stream if isinstance(stream, torch.cuda.Stream) else torch.cuda.ExternalStream(stream.cuda_stream))


def _empty(stream):
    """torch.empty for a call's results on `stream` (None: the current one)."""
    if stream is None:
        return torch.empty

    def empty(*shape, dtype, device):
        with _own(stream):
            t = torch.empty(*shape, dtype=dtype, device=device)
        t.record_stream(torch.cuda.current_stream(device))   # (read there: used again only after that)
        return t
    return empty


def _cuda(t: torch.Tensor, name: str) -> torch.Tensor:
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor")
    return t


# ---------------------------------------------------------------- sizes

def packed_bytes_q4(K: int, N: int) -> int:
    return int(lib().nq_packed_bytes_q4(K, N))


def packed_bytes_q5(K: int, N: int) -> int:
    return int(lib().nq_packed_bytes_q5(K, N))


def scale_bytes(K: int, N: int) -> int:
    return int(lib().nq_scale_bytes(K, N))


# ---------------------------------------------------------------- repack

def _packed_pair(code_bytes: int, K: int, N: int, dev, stream):
    empty = _empty(stream)
    wq = empty(max(code_bytes, 16), dtype=torch.uint8, device=dev)
    s = empty(max(scale_bytes(K, N), 16), dtype=torch.uint8, device=dev)
    return wq, s


def pack_q4(wq_canon: torch.Tensor, s_canon: torch.Tensor, K: int, N: int, stream=None):
    """Canonical Q4 codes (4-byte words [N][K/8]) and fp16 scales ([N][K/64]) on the GPU ->
    (packed codes, packed scales), two uint8 device tensors."""
    dev = _cuda(wq_canon, "wq_canon").device
    _cuda(s_canon, "s_canon")
    wq, s = _packed_pair(packed_bytes_q4(K, N), K, N, dev, stream)
    _check(lib().nq_pack_q4(_ptr(wq_canon), _ptr(s_canon), K, N, _ptr(wq), _ptr(s), _stream(stream)))
    return wq, s


def pack_q5(wn_canon, wh_canon, s_canon, K: int, N: int, stream=None):
    """Canonical Q5 nibble plane, high plane and fp16 scales -> (packed codes, packed scales)."""
    dev = _cuda(wn_canon, "wn_canon").device
    _cuda(wh_canon, "wh_canon")
    _cuda(s_canon, "s_canon")
    wq, s = _packed_pair(packed_bytes_q5(K, N), K, N, dev, stream)
    _check(lib().nq_pack_q5(_ptr(wn_canon), _ptr(wh_canon), _ptr(s_canon), K, N, _ptr(wq), _ptr(s),
                            _stream(stream)))
    return wq, s


# ---------------------------------------------------------------- projections

def _out(x: torch.Tensor, N: int, out, stream=None):
    T = x.shape[0]
    if out is None:
        out = _empty(stream)((T, N), dtype=torch.bfloat16, device=x.device)
    return _cuda(out, "out")


def gemm_q4(x: torch.Tensor, wq: torch.Tensor, s: torch.Tensor, N: int, out=None, stream=None):
    """Y[T,N] (bf16) = X[T,K] (bf16) * dequant(packed Q4 codes wq, packed scales s)."""
    _cuda(x, "x")
    T, K = x.shape
    y = _out(x, N, out, stream)
    _check(lib().nq_gemm_q4(_ptr(x), _ptr(wq), _ptr(s), _ptr(y), T, K, N, _stream(stream)))
    return y


def gemm_q5(x: torch.Tensor, wq: torch.Tensor, s: torch.Tensor, N: int, out=None, stream=None):
    """Y[T,N] (bf16) = X[T,K] (bf16) * dequant(packed Q5 codes wq, packed scales s)."""
    _cuda(x, "x")
    T, K = x.shape
    y = _out(x, N, out, stream)
    _check(lib().nq_gemm_q5(_ptr(x), _ptr(wq), _ptr(s), _ptr(y), T, K, N, _stream(stream)))
    return y


def gemm_q4_noalloc(x: torch.Tensor, wq: torch.Tensor, s: torch.Tensor, N: int, out=None, stream=None):
    """gemm_q4 with its scratch in the library's fixed device array (no allocation by the
    library; `out` is allocated here by torch when not given)."""
    _cuda(x, "x")
    T, K = x.shape
    y = _out(x, N, out, stream)
    _check(lib().nq_gemm_q4_noalloc(_ptr(x), _ptr(wq), _ptr(s), _ptr(y), T, K, N, _stream(stream)))
    return y


def _grouped(fn, x, groups, outs, stream):
    _cuda(x, "x")
    T, K = x.shape
    if outs is None:
        empty = _empty(stream)
        outs = [empty((T, N), dtype=torch.bfloat16, device=x.device) for (_, _, N) in groups]
    arr = (NqGroup * len(groups))()
    for i, ((wq, s, N), y) in enumerate(zip(groups, outs)):
        _cuda(y, "out")
        arr[i] = NqGroup(wq.data_ptr(), s.data_ptr(), y.data_ptr(), N)
    _check(fn(_ptr(x), ctypes.cast(arr, ctypes.c_void_p), len(groups), T, K, _stream(stream)))
    return outs


def gemm_q4_grouped(x, groups, outs=None, stream=None):
    """[Y_g] for groups [(packed codes, packed scales, N_g), ...] sharing X, one launch."""
    return _grouped(lib().nq_gemm_q4_grouped, x, groups, outs, stream)


def gemm_q5_grouped(x, groups, outs=None, stream=None):
    return _grouped(lib().nq_gemm_q5_grouped, x, groups, outs, stream)


def swiglu_q4(x, wg, sg, wu, su, N: int, out=None, stream=None):
    """H[T,N] = bf16(silu(X*Wg) * (X*Wu)) with both weights packed Q4 (codes, scales)."""
    _cuda(x, "x")
    T, K = x.shape
    h = _out(x, N, out, stream)
    _check(lib().nq_swiglu_q4(_ptr(x), _ptr(wg), _ptr(sg), _ptr(wu), _ptr(su), _ptr(h), T, K, N,
                              _stream(stream)))
    return h


def swiglu_q5(x, wg, sg, wu, su, N: int, out=None, stream=None):
    """H[T,N] = bf16(silu(X*Wg) * (X*Wu)) with both weights packed Q5 (codes, scales)."""
    _cuda(x, "x")
    T, K = x.shape
    h = _out(x, N, out, stream)
    _check(lib().nq_swiglu_q5(_ptr(x), _ptr(wg), _ptr(sg), _ptr(wu), _ptr(su), _ptr(h), T, K, N,
                              _stream(stream)))
    return h


def _dequant(fn, wq, s, K: int, N: int, stream):
    out = _empty(stream)((N, K), dtype=torch.float32, device=wq.device)
    _check(fn(_ptr(wq), _ptr(s), _ptr(out), K, N, _stream(stream)))
    return out


def dequant_q4_debug(wq, s, K: int, N: int, operands: str = "f16", stream=None) -> torch.Tensor:
    """fp32 [N][K] dump of a packed Q4 pair through the decoder of the fp16-operand kernels
    (T <= 2, operands="f16") or of the bf16-operand kernels (T >= 3, operands="bf16")."""
    f = lib().nq_dequant_q4_debug if operands == "f16" else lib().nq_dequant_q4_debug_bf16
    return _dequant(f, wq, s, K, N, stream)


def dequant_q5_debug(wq, s, K: int, N: int, operands: str = "f16", stream=None) -> torch.Tensor:
    f = lib().nq_dequant_q5_debug if operands == "f16" else lib().nq_dequant_q5_debug_bf16
    return _dequant(f, wq, s, K, N, stream)


# ---------------------------------------------------------------- NVFP4

def packed_bytes_fp4(K: int, N: int) -> int:
    return int(lib().nq_packed_bytes_fp4(K, N))


def scale_bytes_fp4(K: int, N: int) -> int:
    return int(lib().nq_scale_bytes_fp4(K, N))


def pack_fp4(codes_canon: torch.Tensor, sf_canon: torch.Tensor, K: int, N: int, stream=None):
    """Canonical NVFP4 codes (4-byte words [N][K/8]) and e4m3 scales (bytes [N][K/16]) on the
    GPU -> (packed codes, packed scales), two uint8 device tensors."""
    dev = _cuda(codes_canon, "codes_canon").device
    _cuda(sf_canon, "sf_canon")
    empty = _empty(stream)
    wq = empty(max(packed_bytes_fp4(K, N), 16), dtype=torch.uint8, device=dev)
    s = empty(max(scale_bytes_fp4(K, N), 16), dtype=torch.uint8, device=dev)
    _check(lib().nq_pack_fp4(_ptr(codes_canon), _ptr(sf_canon), K, N, _ptr(wq), _ptr(s), _stream(stream)))
    return wq, s


def gemm_fp4(x: torch.Tensor, wq: torch.Tensor, s: torch.Tensor, global_scale: float, N: int, out=None,
             stream=None):
    """Y[T,N] (bf16) = X[T,K] (bf16) * NVFP4 weight (packed codes wq, packed scales s, tensor
    scale global_scale)."""
    _cuda(x, "x")
    T, K = x.shape
    y = _out(x, N, out, stream)
    _check(lib().nq_gemm_fp4(_ptr(x), _ptr(wq), _ptr(s), ctypes.c_float(global_scale), _ptr(y), T, K, N,
                             _stream(stream)))
    return y


def swiglu_fp4(x, wg, sg, gate_scale: float, wu, su, up_scale: float, N: int, out=None, stream=None):
    """H[T,N] = bf16(silu(X*Wg) * (X*Wu)) with NVFP4 gate and up weights (packed codes, packed
    scales, tensor scale each)."""
    _cuda(x, "x")
    T, K = x.shape
    h = _out(x, N, out, stream)
    _check(lib().nq_swiglu_fp4(_ptr(x), _ptr(wg), _ptr(sg), ctypes.c_float(gate_scale), _ptr(wu), _ptr(su),
                               ctypes.c_float(up_scale), _ptr(h), T, K, N, _stream(stream)))
    return h


def dequant_fp4_debug(wq, s, global_scale: float, K: int, N: int, stream=None) -> torch.Tensor:
    out = _empty(stream)((N, K), dtype=torch.float32, device=wq.device)
    _check(lib().nq_dequant_fp4_debug(_ptr(wq), _ptr(s), ctypes.c_float(global_scale), _ptr(out), K, N,
                                      _stream(stream)))
    return out


# ---------------------------------------------------------------- recorded programs

PROGRAM_KEYS = ("calls", "kernels", "builds", "failed_call")


class Program:
    """A sequence of projection calls recorded once and replayed as one CUDA graph
    (nq_program_* of include/nq.h). The library records the tensors' device addresses, not
    their contents: write new activations into the same X tensor and launch again. The
    program keeps a reference to every tensor it records, so they stay allocated while it can
    be launched. Outputs not given are allocated here (torch) and returned."""

    def __init__(self):
        h = ctypes.c_void_p()
        _check(lib().nq_program_create(ctypes.byref(h)))
        self._h = h
        self._keep = []

    def _rec(self, status, *tensors):
        _check(status)
        self._keep.extend(t for t in tensors if t is not None)

    def _gemm(self, bits, x, wq, s, N, out):
        _cuda(x, "x")
        T, K = x.shape
        y = _out(x, N, out)
        self._rec(lib().nq_program_gemm(self._h, bits, _ptr(x), _ptr(wq), _ptr(s), _ptr(y), T, K, N), x, wq, s, y)
        return y

    def gemm_q4(self, x, wq, s, N: int, out=None):
        return self._gemm(4, x, wq, s, N, out)

    def gemm_q5(self, x, wq, s, N: int, out=None):
        return self._gemm(5, x, wq, s, N, out)

    def gemm_fp4(self, x, wq, s, global_scale: float, N: int, out=None):
        _cuda(x, "x")
        T, K = x.shape
        y = _out(x, N, out)
        self._rec(lib().nq_program_gemm_fp4(self._h, _ptr(x), _ptr(wq), _ptr(s), ctypes.c_float(global_scale),
                                            _ptr(y), T, K, N), x, wq, s, y)
        return y

    def _swiglu(self, bits, x, wg, sg, wu, su, N, out):
        _cuda(x, "x")
        T, K = x.shape
        h = _out(x, N, out)
        self._rec(lib().nq_program_swiglu(self._h, bits, _ptr(x), _ptr(wg), _ptr(sg), _ptr(wu), _ptr(su), _ptr(h),
                                          T, K, N), x, wg, sg, wu, su, h)
        return h

    def swiglu_q4(self, x, wg, sg, wu, su, N: int, out=None):
        return self._swiglu(4, x, wg, sg, wu, su, N, out)

    def swiglu_q5(self, x, wg, sg, wu, su, N: int, out=None):
        return self._swiglu(5, x, wg, sg, wu, su, N, out)

    def swiglu_fp4(self, x, wg, sg, gate_scale: float, wu, su, up_scale: float, N: int, out=None):
        _cuda(x, "x")
        T, K = x.shape
        h = _out(x, N, out)
        self._rec(lib().nq_program_swiglu_fp4(self._h, _ptr(x), _ptr(wg), _ptr(sg), ctypes.c_float(gate_scale),
                                              _ptr(wu), _ptr(su), ctypes.c_float(up_scale), _ptr(h), T, K, N),
                  x, wg, sg, wu, su, h)
        return h

    def _grouped(self, bits, x, groups, outs):
        _cuda(x, "x")
        T, K = x.shape
        if outs is None:
            outs = [torch.empty((T, N), dtype=torch.bfloat16, device=x.device) for (_, _, N) in groups]
        arr = (NqGroup * len(groups))()
        for i, ((wq, s, N), y) in enumerate(zip(groups, outs)):
            _cuda(y, "out")
            arr[i] = NqGroup(wq.data_ptr(), s.data_ptr(), y.data_ptr(), N)
        self._rec(lib().nq_program_grouped(self._h, bits, _ptr(x), ctypes.cast(arr, ctypes.c_void_p), len(groups),
                                           T, K), x, *[t for (wq, s, _) in groups for t in (wq, s)], *outs)
        return outs

    def grouped_q4(self, x, groups, outs=None):
        return self._grouped(4, x, groups, outs)

    def grouped_q5(self, x, groups, outs=None):
        return self._grouped(5, x, groups, outs)

    def build(self) -> None:
        _check(lib().nq_program_build(self._h))

    def launch(self, stream=None) -> None:
        _check(lib().nq_program_launch(self._h, _stream(stream)))

    def info(self) -> dict:
        out = (ctypes.c_int64 * 4)()
        _check(lib().nq_program_info(self._h, ctypes.cast(out, ctypes.c_void_p)))
        return dict(zip(PROGRAM_KEYS, list(out)))

    def close(self) -> None:
        if self._h is not None and self._h.value:
            lib().nq_program_destroy(self._h)
        self._h = None
        self._keep = []

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass


# ---------------------------------------------------------------- serving step

# These calls are short (a few microseconds on the GPU), so the checks here touch each tensor as
# little as they can.

_DTYPES = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
_KV = struct.Struct("PPqqqiiii")    # struct nq_kv_cache


def _raw_stream(stream) -> int:
    """The stream's handle; None: the current stream of the current device."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _flat(t, name: str, dtype, n: int) -> int:
    """The address of a contiguous CUDA tensor of n elements."""
    try:
        if t.dtype is dtype and t.numel() == n and t.is_cuda and t.is_contiguous():
            return t.data_ptr()
    except AttributeError:
        pass
    raise ValueError(f"{name} must be a contiguous CUDA tensor of {n} elements of {dtype}")


def _rows(t, name: str, dtype, rows: int):
    """(address, columns, stride between rows) of a CUDA tensor [rows][columns], its rows contiguous."""
    try:
        if t.dtype is dtype and t.is_cuda:
            n, cols = t.shape
            stride, one = t.stride()
            if n == rows and (one == 1 or cols <= 1 or n == 0):
                return t.data_ptr(), cols, stride if n > 1 else max(cols, 1)
    except (AttributeError, ValueError):
        pass
    raise ValueError(f"{name} must be a CUDA tensor of {dtype} with {rows} rows, each contiguous")


def _tokens(t, name: str, dtype, heads, dim):
    """(address, tokens, heads, stride between tokens) of a CUDA tensor [tokens][heads][dim] whose
    token rows lie together; heads None: any."""
    try:
        if t.dtype is dtype and t.is_cuda:
            n, h, d = t.shape
            st, sh, sd = t.stride()
            if d == dim and (heads is None or h == heads) and sd == 1 and (sh == dim or h <= 1):
                return t.data_ptr(), n, h, st if n > 1 else h * dim
    except (AttributeError, ValueError):
        pass
    raise ValueError(f"{name} must be a CUDA tensor of {dtype}, [tokens][{heads or 'heads'}][{dim}] with contiguous "
                     "token rows")


def _kv_cache(k_cache, v_cache):
    """(struct nq_kv_cache, dtype, heads, dim) of a paged cache given as two
    [num_blocks][page][heads][dim] tensors of equal strides (for a cache stored
    [num_blocks][heads][page][dim], pass cache.transpose(1, 2))."""
    try:
        dt = k_cache.dtype
        if (dt is torch.bfloat16 or dt is torch.float16) and v_cache.dtype is dt and k_cache.is_cuda and v_cache.is_cuda:
            shape, strides = k_cache.shape, k_cache.stride()
            blocks, page, heads, dim = shape
            bs, rs, hs, ds = strides
            if ds == 1 and v_cache.shape == shape and v_cache.stride() == strides:
                # the stride of a dimension of one element means nothing
                return (_KV.pack(k_cache.data_ptr(), v_cache.data_ptr(), bs if blocks > 1 else max(bs, dim), rs,
                                 hs if heads > 1 else dim, blocks, page, heads, dim), dt, heads, dim)
    except (AttributeError, ValueError):
        pass
    raise ValueError("k_cache and v_cache must be CUDA tensors [num_blocks][page][heads][dim] of bfloat16 or float16 "
                     "with one shape, the same strides and contiguous last dimensions")


def page_tables(lens, new_lens, free_blocks, num_free, block_table, page: int, max_tokens: int, out=None, stream=None):
    """Block tables and slot maps of a step from the requests' lengths (nq_page_tables): extends
    block_table in place from the free list and returns (q_start [R+1], kv_lens [R],
    positions [max_tokens], slots [max_tokens], counts [3]: tokens, blocks taken, requests
    refused). All tensors int32 on the GPU (slots int64); `out`: the five outputs, to be reused."""
    i32 = torch.int32
    R = lens.numel()
    table, max_blocks, stride = _rows(block_table, "block_table", i32, R)
    if out is None:
        dev, empty = lens.device, _empty(stream)
        out = (empty(R + 1, dtype=i32, device=dev), empty(R, dtype=i32, device=dev),
               empty(max_tokens, dtype=i32, device=dev), empty(max_tokens, dtype=torch.int64, device=dev),
               empty(3, dtype=i32, device=dev))
    q_start, kv_lens, positions, slots, counts = out
    free = free_blocks.numel()
    _check(lib().nq_page_tables(_flat(lens, "lens", i32, R), _flat(new_lens, "new_lens", i32, R), R,
                                _flat(free_blocks, "free_blocks", i32, free), free, _flat(num_free, "num_free", i32, 1),
                                page, table, stride, max_blocks, _flat(q_start, "q_start", i32, R + 1),
                                _flat(kv_lens, "kv_lens", i32, R), _flat(positions, "positions", i32, max_tokens),
                                _flat(slots, "slots", torch.int64, max_tokens), max_tokens,
                                _flat(counts, "counts", i32, 3), _raw_stream(stream)))
    return out


def kv_append(k, v, slots, k_cache, v_cache, stream=None) -> None:
    """Store new keys and values [tokens][heads][dim] at slots [tokens] (int64; block * page + row,
    -1 for none) of the paged cache [num_blocks][page][heads][dim] (nq_kv_append)."""
    cache, dt, heads, dim = _kv_cache(k_cache, v_cache)
    kp, tokens, _, ks = _tokens(k, "k", dt, heads, dim)
    vp, tokens_v, _, vs = _tokens(v, "v", dt, heads, dim)
    if tokens_v != tokens:
        raise ValueError("k and v must have the same number of tokens")
    _check(lib().nq_kv_append(kp, ks, vp, vs, _flat(slots, "slots", torch.int64, tokens), tokens, cache,
                              _raw_stream(stream)))


def attn_paged(q, k_cache, v_cache, block_table, q_start, kv_lens, scale: float = None, window: int = 0,
               sinks: int = 0, out=None, stream=None):
    """Causal attention of a step's new tokens q [tokens][q_heads][dim] over the paged cache
    [num_blocks][page][heads][dim] (nq_attn_paged): block_table [R][max_blocks], q_start [R+1]
    and kv_lens [R] (int32, as page_tables gives them). scale defaults to dim ** -0.5; window > 0
    limits a token to the last `window` keys and the first `sinks`. Returns out [tokens][q_heads][dim]."""
    cache, dt, _, dim = _kv_cache(k_cache, v_cache)
    qp, tokens, heads, qs = _tokens(q, "q", dt, None, dim)
    if out is None:
        out = _empty(stream)((tokens, heads, dim), dtype=dt, device=q.device)
    op, tokens_o, _, os_ = _tokens(out, "out", dt, heads, dim)
    if tokens_o != tokens:
        raise ValueError("out must have q's shape")
    R = kv_lens.numel()
    table, max_blocks, stride = _rows(block_table, "block_table", torch.int32, R)
    _check(lib().nq_attn_paged(qp, qs, cache, table, stride, max_blocks, _flat(q_start, "q_start", torch.int32, R + 1),
                               _flat(kv_lens, "kv_lens", torch.int32, R), R, tokens, heads,
                               dim ** -0.5 if scale is None else scale, window, sinks, _DTYPES[dt], op, os_,
                               _raw_stream(stream)))
    return out


def attn_reserve() -> None:
    """Allocate the attention workspace now (before stream capture)."""
    _check(lib().nq_attn_reserve())


def sample(logits, noise, temperature=None, top_k=None, top_p=None, min_p=None, out=None, stream=None):
    """The next token of each row of logits [B][V] (bfloat16, float16 or float32) with the row's
    temperature, top_k, top_p and min_p ([B] tensors, None for none) and noise [B][V] (float32,
    independent Exp(1) variates: `torch.empty_like(...).exponential_()`); see nq_sample. Returns
    int32 tokens [B], -1 for a row without a candidate."""
    dtype = _DTYPES.get(logits.dtype)
    if dtype is None:
        raise ValueError("logits must be bfloat16, float16 or float32")
    B, f32 = logits.shape[0], torch.float32
    lp, V, stride = _rows(logits, "logits", logits.dtype, B)
    np_, V_noise, noise_stride = _rows(noise, "noise", f32, B)
    if V_noise != V:
        raise ValueError("noise must have the shape of logits")
    if out is None:
        out = _empty(stream)(B, dtype=torch.int32, device=logits.device)
    _check(lib().nq_sample(lp, dtype, stride, np_, noise_stride, B, V,
                           None if temperature is None else _flat(temperature, "temperature", f32, B),
                           None if top_k is None else _flat(top_k, "top_k", torch.int32, B),
                           None if top_p is None else _flat(top_p, "top_p", f32, B),
                           None if min_p is None else _flat(min_p, "min_p", f32, B),
                           _flat(out, "out", torch.int32, B), _raw_stream(stream)))
    return out


# ---------------------------------------------------------------- 8-bit products and experts

_E4M3 = torch.float8_e4m3fn
_F8_ROWS = struct.Struct("PPqqi4x")      # struct nq_fp8_rows
_F8_WEIGHT = struct.Struct("PPqqqq")     # struct nq_fp8_weight
_F8_OUT = struct.Struct("PPqqi4x")       # struct nq_fp8_out
_F8_DTYPES = {torch.bfloat16: 0, torch.float16: 1, _E4M3: 3}
_SCORES = {"softmax": 0, "sigmoid": 1}


def quant_fp8(x, out=None, stream=None):
    """x [rows][K] (bfloat16, float16 or float32) as e4m3 codes [rows][K] and float32 scales
    [rows][ceil(K / 128)], one for each 128 columns of a row (nq_quant_fp8). `out`: (codes, scales), to be reused."""
    dtype = _DTYPES.get(x.dtype)
    if dtype is None:
        raise ValueError("x must be bfloat16, float16 or float32")
    rows = x.shape[0]
    xp, K, stride = _rows(x, "x", x.dtype, rows)
    if out is None:
        empty = _empty(stream)
        out = (empty((rows, K), dtype=_E4M3, device=x.device),
               empty((rows, -(-K // 128)), dtype=torch.float32, device=x.device))
    codes, scales = out
    cp, K_c, cs = _rows(codes, "codes", _E4M3, rows)
    sp, blocks, ss = _rows(scales, "scales", torch.float32, rows)
    if K_c != K or blocks != -(-K // 128):
        raise ValueError("codes must have x's shape and scales a column for each 128 of it")
    _check(lib().nq_quant_fp8(xp, dtype, stride, rows, K, cp, cs, sp, ss, _raw_stream(stream)))
    return out


def _fp8_weight(codes, scales, E, name: str):
    """(struct nq_fp8_weight, N, K) of codes [N][K] and scales [ceil(N / 128)][ceil(K / 128)], with experts (E not
    None) [E][..][..] both."""
    try:
        if codes.dtype is _E4M3 and scales.dtype is torch.float32 and codes.is_cuda and scales.is_cuda:
            shape, block, st, ss = codes.shape, scales.shape, codes.stride(), scales.stride()
            if E is None:
                (N, K), (nb, kb), e, se = shape, block, 0, 0
            else:
                (n, N, K), (m, nb, kb), e, se = shape, block, st[0], ss[0]
                if n != E or m != E:
                    raise ValueError
            if nb == -(-N // 128) and kb == -(-K // 128) and (st[-1] == 1 or K <= 1) and (ss[-1] == 1 or kb <= 1):
                return _F8_WEIGHT.pack(codes.data_ptr(), scales.data_ptr(), st[-2], e, ss[-2], se), N, K
    except (AttributeError, ValueError):
        pass
    raise ValueError(f"{name} must be CUDA tensors of float8_e4m3fn codes {'' if E is None else '[experts]'}[N][K] and float32 "
                     "scales, one for each 128 x 128, contiguous along K")


def _fp8(fn, xq, xs, weights, dtype, out, stream, experts=None):
    """The four products; experts: (offsets, rows)."""
    x_rows = xq.shape[0]
    xp, K, stride = _rows(xq, "xq", _E4M3, x_rows)
    sp, kb, ss = _rows(xs, "xs", torch.float32, x_rows)
    E, M = None, x_rows
    if experts is not None:
        offsets, rows = experts
        E = offsets.numel() - 1
        offsets = _flat(offsets, "offsets", torch.int32, E + 1)
        if rows is not None:
            M = rows.numel()
            rows = _flat(rows, "rows", torch.int32, M)
    packed = []
    for codes, scales in weights:
        w, N, K_w = _fp8_weight(codes, scales, E, "the weights")
        if K_w != K or (packed and N != width):
            raise ValueError("the weights must have xq's K, and the same N")
        width = N
        packed.append(w)
    if kb != -(-K // 128):
        raise ValueError("xs must have a column for each 128 of xq")
    if out is None:
        empty = _empty(stream)
        out = empty((M, N), dtype=dtype, device=xq.device)
        if dtype is _E4M3:
            out = (out, empty((M, -(-N // 128)), dtype=torch.float32, device=xq.device))
    if dtype is _E4M3:
        yp, N_y, ys = _rows(out[0], "out", dtype, M)
        yc, nb, yss = _rows(out[1], "out's scales", torch.float32, M)
        if nb != -(-N // 128):
            raise ValueError("out's scales must have a column for each 128 of it")
    else:
        yp, N_y, ys = _rows(out, "out", dtype, M)
        yc = yss = 0
    if N_y != N:
        raise ValueError("out must have a column for each row of the weights")
    x = _F8_ROWS.pack(xp, sp, stride, ss, x_rows)
    y = _F8_OUT.pack(yp, yc, ys, yss, _F8_DTYPES.get(dtype, -1))
    if experts is None:
        _check(fn(x, *packed, y, K, N, _raw_stream(stream)))
    else:
        need = lib().nq_fp8_scratch_bytes(M, E, K, len(packed) - 1) if rows is not None else 0
        if need:
            if stream is None:
                scratch = torch.empty(need, dtype=torch.uint8, device=xq.device)
            else:                                # (used there alone)
                with _own(stream):
                    scratch = torch.empty(need, dtype=torch.uint8, device=xq.device)
        _check(fn(x, rows, M, offsets, E, *packed, y, K, N, scratch.data_ptr() if need else None, _raw_stream(stream)))
    return out


def gemm_fp8(xq, xs, wq, ws, dtype=torch.bfloat16, out=None, stream=None):
    """y [rows][N] (bfloat16 or float16) = x w^T of e4m3 codes with block scales (nq_gemm_fp8): xq [rows][K] with
    float32 xs [rows][ceil(K / 128)] (quant_fp8), wq [N][K] with ws [ceil(N / 128)][ceil(K / 128)]."""
    return _fp8(lib().nq_gemm_fp8, xq, xs, ((wq, ws),), dtype, out, stream)


def swiglu_fp8(xq, xs, wg, sg, wu, su, dtype=torch.bfloat16, out=None, stream=None):
    """silu(x wg^T) * (x wu^T), weights as in gemm_fp8 (nq_swiglu_fp8). dtype float8_e4m3fn returns (codes, scales), quantised
    as quant_fp8 does: what the down projection takes."""
    return _fp8(lib().nq_swiglu_fp8, xq, xs, ((wg, sg), (wu, su)), dtype, out, stream)


def gemm_fp8_experts(xq, xs, wq, ws, offsets, rows=None, dtype=torch.bfloat16, out=None, stream=None):
    """gemm_fp8 with a weight for each expert: row i, offsets[e] <= i < offsets[e + 1] (int32 [E + 1], on the GPU),
    is row rows[i] of x (int32; None: i) times wq[e] [E][N][K] with ws [E][..][..] (nq_gemm_fp8_experts)."""
    return _fp8(lib().nq_gemm_fp8_experts, xq, xs, ((wq, ws),), dtype, out, stream, (offsets, rows))


def swiglu_fp8_experts(xq, xs, wg, sg, wu, su, offsets, rows=None, dtype=torch.bfloat16, out=None, stream=None):
    """swiglu_fp8 with gate and up weights for each expert, rows as in gemm_fp8_experts (nq_swiglu_fp8_experts)."""
    return _fp8(lib().nq_swiglu_fp8_experts, xq, xs, ((wg, sg), (wu, su)), dtype, out, stream, (offsets, rows))


def moe_route(logits, k: int, bias=None, score: str = "softmax", normalize: bool = True, scale: float = 1.0, out=None,
              stream=None):
    """Each token's k experts from logits [T][E] (nq_moe_route). score "softmax" or "sigmoid"; bias float32 [E]
    (sigmoid: choose by score + bias); normalize: the weights sum to `scale`. Returns (ids [T][k], weights [T][k] float32, offsets
    [E + 1], rows [T * k], slots [T][k]), int32: `out`, to be reused."""
    dtype = _DTYPES.get(logits.dtype)
    if dtype is None or score not in _SCORES:
        raise ValueError("logits must be bfloat16, float16 or float32, and score softmax or sigmoid")
    T, i32 = logits.shape[0], torch.int32
    lp, E, stride = _rows(logits, "logits", logits.dtype, T)
    if out is None:
        dev, empty = logits.device, _empty(stream)
        out = (empty((T, k), dtype=i32, device=dev), empty((T, k), dtype=torch.float32, device=dev),
               empty(E + 1, dtype=i32, device=dev), empty(T * k, dtype=i32, device=dev),
               empty((T, k), dtype=i32, device=dev))
    ids, weights, offsets, rows, slots = out
    n = T * k
    _check(lib().nq_moe_route(lp, dtype, stride, None if bias is None else _flat(bias, "bias", torch.float32, E), T, E, k,
                              _SCORES[score], int(normalize), scale, _flat(ids, "ids", i32, n),
                              _flat(weights, "weights", torch.float32, n), _flat(offsets, "offsets", i32, E + 1),
                              _flat(rows, "rows", i32, n), _flat(slots, "slots", i32, n), _raw_stream(stream)))
    return out


def moe_combine(y, slots, weights, base=None, out=None, stream=None):
    """out [T][N] = base + sum_j weights[:, j] * y[slots[:, j]] (nq_moe_combine): y [rows][N] (bfloat16 or
    float16), slots int32 and weights float32 [T][k] as moe_route gives them, base [T][N] or None. out may be base."""
    dt = y.dtype
    if dt is not torch.bfloat16 and dt is not torch.float16:
        raise ValueError("y must be bfloat16 or float16")
    T, k = slots.shape
    M = y.shape[0]
    yp, N, ys = _rows(y, "y", dt, M)
    bp, bs = None, 0
    if base is not None:
        bp, N_b, bs = _rows(base, "base", dt, T)
        if N_b != N:
            raise ValueError("base must have y's columns")
    if out is None:
        out = _empty(stream)((T, N), dtype=dt, device=y.device)
    op, N_o, os_ = _rows(out, "out", dt, T)
    if N_o != N:
        raise ValueError("out must have y's columns")
    _check(lib().nq_moe_combine(yp, _DTYPES[dt], ys, M, _flat(slots, "slots", torch.int32, T * k),
                                _flat(weights, "weights", torch.float32, T * k), T, k, N, bp, bs, op, os_,
                                _raw_stream(stream)))
    return out


# ---------------------------------------------------------------- runtime / plan

def reserve(T_max: int, K_max: int, N_max: int) -> None:
    _check(lib().nq_reserve(T_max, K_max, N_max))


def device_error() -> None:
    _check(lib().nq_device_error())


def wait_limit(ns: int = 0) -> int:
    """Set (ns > 0) or query (ns <= 0) the bound of device-side waits; returns the previous."""
    return int(lib().nq_wait_limit(int(ns)))


def shutdown() -> None:
    lib().nq_shutdown()


PLAN_KEYS = ("ctas", "units", "slabs", "slab_groups", "pairs", "ws_slots", "stages", "chunk_groups")


def plan_info(bits: int, mode: int, T: int, K: int, N: int, num_sms: int) -> dict:
    out = (ctypes.c_int64 * 8)()
    _check(lib().nq_plan_info(bits, mode, T, K, N, num_sms, ctypes.cast(out, ctypes.c_void_p)))
    return dict(zip(PLAN_KEYS, list(out)))


def plan_segments(bits: int, mode: int, T: int, K: int, N: int, num_sms: int, cta: int) -> list:
    n = lib().nq_plan_segments(bits, mode, T, K, N, num_sms, cta, None, 0)
    if n < 0:
        _check(int(n))
    buf = (ctypes.c_int64 * (4 * max(n, 1)))()
    lib().nq_plan_segments(bits, mode, T, K, N, num_sms, cta, ctypes.cast(buf, ctypes.c_void_p), n)
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(n)]


def tensor_core_batches(enable: int = -1) -> int:
    """Large batches (8 < T <= 64) on the tensor-core kernel (1) or in 8-token slices (0); -1
    queries. Returns the previous setting."""
    return int(lib().nq_tensor_core_batches(enable))


TC_KEYS = ("ctas", "row_blocks", "k_pieces", "tokens_padded", "stages", "smem_bytes", "groups", "stage_groups")


def plan_tc_info(bits: int, T: int, K: int, N: int, num_sms: int) -> dict:
    out = (ctypes.c_int64 * 8)()
    _check(lib().nq_plan_tc_info(bits, T, K, N, num_sms, ctypes.cast(out, ctypes.c_void_p)))
    return dict(zip(TC_KEYS, list(out)))


ROUTE_KEYS = ("kernel", "launches", "operands", "split", "ctas", "k_split", "stages", "tokens_padded")
ROUTE_NAMES = {"kernel": ("mma.sync 8-token", "tcgen05"), "operands": ("fp16", "bf16"),
               "split": ("stream-K", "whole row pairs", "slab clusters", "row blocks x K pieces")}


def route_info(bits: int, mode: int, T: int, K: int, N: int, num_sms: int) -> dict:
    """The kernel and variant a call of this shape takes with the current settings (host
    only): ROUTE_KEYS, with the kernel, operand type and split also given by name."""
    out = (ctypes.c_int64 * 8)()
    _check(lib().nq_route_info(bits, mode, T, K, N, num_sms, ctypes.cast(out, ctypes.c_void_p)))
    d = dict(zip(ROUTE_KEYS, list(out)))
    for k, names in ROUTE_NAMES.items():
        d[k + "_name"] = names[d[k]]
    return d


def slab_clusters(enable: int = -1) -> int:
    """Turn slab clusters on (1) / off (0) for later calls, or query (-1); returns the
    previous setting."""
    return int(lib().nq_slab_clusters(enable))


CLUSTER_KEYS = ("ctas", "cluster", "slab_groups", "pairs", "ws_slots", "stages", "cluster_units", "clusters")


def plan_cluster_info(bits: int, mode: int, T: int, K: int, N: int, clusters: int) -> dict:
    """The slab-cluster plan of a shape (host only); raises NqError if the shape has none."""
    out = (ctypes.c_int64 * 8)()
    _check(lib().nq_plan_cluster_info(bits, mode, T, K, N, clusters, ctypes.cast(out, ctypes.c_void_p)))
    return dict(zip(CLUSTER_KEYS, list(out)))


def plan_cluster_segments(bits: int, mode: int, T: int, K: int, N: int, clusters: int, cta: int):
    """Real (slab, pair, ga, gb) runs of block `cta` of a slab-cluster plan, in order."""
    n = lib().nq_plan_cluster_segments(bits, mode, T, K, N, clusters, cta, None, 0)
    if n < 0:
        _check(int(n))
    buf = (ctypes.c_int64 * (4 * max(n, 1)))()
    lib().nq_plan_cluster_segments(bits, mode, T, K, N, clusters, cta, ctypes.cast(buf, ctypes.c_void_p), n)
    return [tuple(buf[4 * i:4 * i + 4]) for i in range(n)]


# C names, for callers that prefer them
nq_pack_q4, nq_pack_q5 = pack_q4, pack_q5
nq_gemm_q4, nq_gemm_q5, nq_gemm_q4_noalloc = gemm_q4, gemm_q5, gemm_q4_noalloc
nq_swiglu_q4, nq_swiglu_q5 = swiglu_q4, swiglu_q5
nq_gemm_q4_grouped, nq_gemm_q5_grouped = gemm_q4_grouped, gemm_q5_grouped
nq_dequant_q4_debug, nq_dequant_q5_debug = dequant_q4_debug, dequant_q5_debug
nq_pack_fp4, nq_gemm_fp4, nq_dequant_fp4_debug = pack_fp4, gemm_fp4, dequant_fp4_debug
nq_swiglu_fp4 = swiglu_fp4
nq_reserve, nq_device_error, nq_shutdown, nq_wait_limit = reserve, device_error, shutdown, wait_limit
nq_plan_info, nq_plan_segments = plan_info, plan_segments
nq_page_tables, nq_kv_append, nq_attn_paged, nq_attn_reserve = page_tables, kv_append, attn_paged, attn_reserve
nq_sample = sample
nq_quant_fp8, nq_gemm_fp8, nq_swiglu_fp8 = quant_fp8, gemm_fp8, swiglu_fp8
nq_gemm_fp8_experts, nq_swiglu_fp8_experts = gemm_fp8_experts, swiglu_fp8_experts
nq_moe_route, nq_moe_combine = moe_route, moe_combine
