"""Where a call's results and scratch memory come from when it is given a stream: that stream's own memory. The current stream's
free memory may still be written by kernels that wait there. Stand-ins for tensors, streams and the library: no GPU."""
import contextlib

import pytest
import torch

from weight_only_groupwise_gb300 import nq

BF16, F32, I32, I64, E4M3 = torch.bfloat16, torch.float32, torch.int32, torch.int64, torch.float8_e4m3fn


class Tensor:
    is_cuda, device = True, "cuda"

    def __init__(self, shape, dtype, owner=None):
        self.shape, self.dtype, self.owner, self.readers = tuple(shape), dtype, owner, []

    def stride(self):
        out = [1]
        for n in self.shape[:0:-1]:
            out.insert(0, out[0] * n)
        return tuple(out)

    def numel(self):
        n = 1
        for k in self.shape:
            n *= k
        return n

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return id(self) * 16

    def record_stream(self, stream):
        self.readers.append(stream)


class Stream:
    def __init__(self, handle):
        self.cuda_stream = handle


class Library:
    """Every call succeeds; sizes that some helpers ask for."""

    def __init__(self):
        self.streams = []

    def __getattr__(self, name):
        if name.startswith(("nq_packed_bytes", "nq_scale_bytes")):
            return lambda K, N: 64
        if name == "nq_fp8_scratch_bytes":
            return lambda *a: 4096

        def call(*args):
            last = args[-1]
            self.streams.append(getattr(last, "value", last))
            return 0
        return call


@pytest.fixture
def made(monkeypatch):
    """All tensors that are made, each with the stream that was current."""
    current, tensors, library = [Stream(1)], [], Library()

    @contextlib.contextmanager
    def on(stream):
        before, current[0] = current[0], stream
        yield
        current[0] = before

    def empty(*shape, dtype, device):
        shape = shape[0] if isinstance(shape[0], (tuple, list, torch.Size)) else shape
        tensors.append(Tensor(shape, dtype, current[0]))
        return tensors[-1]

    for where, name, value in ((torch, "empty", empty), (torch, "Tensor", Tensor), (torch.cuda, "stream", on), (torch.cuda, "Stream", Stream),
                               (torch.cuda, "current_stream", lambda device=None: current[0]), (nq, "lib", lambda: library),
                               (nq, "_raw_stream", lambda s: (s or current[0]).cuda_stream)):
        monkeypatch.setattr(where, name, value)
    return tensors, library, current[0]


def t(*shape, dtype=BF16):
    return Tensor(shape, dtype)


def fp8(T, K):
    return t(T, K, dtype=E4M3), t(T, -(-K // 128), dtype=F32)


def w8(*shape):
    return t(*shape, dtype=E4M3), t(*shape[:-2], -(-shape[-2] // 128), -(-shape[-1] // 128), dtype=F32)


KV = dict(k_cache=t(5, 16, 2, 64), v_cache=t(5, 16, 2, 64))
CALLS = {
    "quant_fp8": lambda **s: nq.quant_fp8(t(3, 256), **s),
    "gemm_fp8": lambda **s: nq.gemm_fp8(*fp8(3, 256), *w8(40, 256), **s),
    "swiglu_fp8": lambda **s: nq.swiglu_fp8(*fp8(3, 256), *w8(40, 256), *w8(40, 256), dtype=E4M3, **s),
    "gemm_fp8_experts": lambda **s: nq.gemm_fp8_experts(*fp8(3, 256), *w8(2, 40, 256), t(3, dtype=I32), rows=t(9, dtype=I32), **s),
    "swiglu_fp8_experts": lambda **s: nq.swiglu_fp8_experts(*fp8(3, 256), *w8(2, 40, 256), *w8(2, 40, 256), t(3, dtype=I32), rows=t(9, dtype=I32),
                                                            dtype=E4M3, **s),
    "moe_route": lambda **s: nq.moe_route(t(3, 8), 2, **s),
    "moe_combine": lambda **s: nq.moe_combine(t(6, 64), t(3, 2, dtype=I32), t(3, 2, dtype=F32), **s),
    "page_tables": lambda **s: nq.page_tables(t(2, dtype=I32), t(2, dtype=I32), t(9, dtype=I32), t(1, dtype=I32), t(2, 4, dtype=I32), 16, 8, **s),
    "attn_paged": lambda **s: nq.attn_paged(t(3, 4, 64), **KV, block_table=t(2, 4, dtype=I32), q_start=t(3, dtype=I32), kv_lens=t(2, dtype=I32), **s),
    "sample": lambda **s: nq.sample(t(3, 100), t(3, 100, dtype=F32), **s),
    "gemm_q4": lambda **s: nq.gemm_q4(t(2, 128), t(64), t(64), 32, **s),
    "gemm_q5": lambda **s: nq.gemm_q5(t(2, 128), t(64), t(64), 32, **s),
    "gemm_q4_noalloc": lambda **s: nq.gemm_q4_noalloc(t(2, 128), t(64), t(64), 32, **s),
    "gemm_fp4": lambda **s: nq.gemm_fp4(t(2, 128), t(64), t(64), 1.0, 32, **s),
    "swiglu_q4": lambda **s: nq.swiglu_q4(t(2, 128), t(64), t(64), t(64), t(64), 32, **s),
    "swiglu_q5": lambda **s: nq.swiglu_q5(t(2, 128), t(64), t(64), t(64), t(64), 32, **s),
    "swiglu_fp4": lambda **s: nq.swiglu_fp4(t(2, 128), t(64), t(64), 1.0, t(64), t(64), 1.0, 32, **s),
    "gemm_q4_grouped": lambda **s: nq.gemm_q4_grouped(t(2, 128), [(t(64), t(64), 32), (t(64), t(64), 16)], **s),
    "pack_q4": lambda **s: nq.pack_q4(t(32, 16), t(32, 2), 128, 32, **s),
    "pack_q5": lambda **s: nq.pack_q5(t(32, 16), t(32, 4), t(32, 2), 128, 32, **s),
    "pack_fp4": lambda **s: nq.pack_fp4(t(32, 16), t(32, 8), 128, 32, **s),
    "dequant_q4_debug": lambda **s: nq.dequant_q4_debug(t(64), t(64), 128, 32, **s),
    "dequant_fp4_debug": lambda **s: nq.dequant_fp4_debug(t(64), t(64), 1.0, 128, 32, **s),
}


@pytest.mark.parametrize("name", CALLS)
def test_memory_is_the_given_streams(name, made):
    tensors, library, current = made
    other = Stream(2)
    result = CALLS[name](stream=other)
    assert library.streams[-1] == 2 and tensors and all(x.owner is other for x in tensors)
    # results are read on the current stream: their memory waits for that before it is used again
    for x in result if isinstance(result, (tuple, list)) else (result,):
        assert x.readers == [current]


@pytest.mark.parametrize("name", CALLS)
def test_memory_is_the_current_streams(name, made):
    tensors, library, current = made
    CALLS[name]()
    assert library.streams[-1] == 1 and tensors and all(x.owner is current and not x.readers for x in tensors)
