"""Calls on a stream that is not the current one and that make their results themselves, while the current stream still writes
memory that it has freed."""
import pytest
import torch

from tests import fp8_ref as ref
from weight_only_groupwise_gb300 import nq

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, ref.E4M3


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_only_groupwise_gb300 import build
    build.build()
    yield
    nq.device_error()


def calls(g):
    (x, xs), (w, ws), (v, vs) = ref.activations(1500, 1024, g), ref.weights(4, 512, 1024, g), ref.weights(4, 512, 1024, g)
    xs *= 2.0 ** -10
    ends = torch.tensor([0, 300, 300, 1000, 1500], dtype=torch.int32, device="cuda")
    rows = torch.randperm(1500, device="cuda", generator=g).to(torch.int32)
    logits = torch.randn((1500, 64), device="cuda", generator=g)
    a = torch.randn((1500, 1024), device="cuda", generator=g).to(BF16)
    slots = torch.randint(-1, 1500, (700, 4), device="cuda", generator=g, dtype=torch.int32)
    weights = torch.rand((700, 4), device="cuda", generator=g)
    noise = torch.empty_like(logits).exponential_(generator=g)
    return {
        "quant": lambda **s: nq.quant_fp8(a, **s),
        "gemm": lambda **s: nq.gemm_fp8(x, xs, w[0], ws[0], **s),
        "swiglu": lambda **s: nq.swiglu_fp8(x, xs, w[0], ws[0], v[0], vs[0], dtype=E4M3, **s),
        "experts": lambda **s: nq.gemm_fp8_experts(x, xs, w, ws, ends, rows=rows, **s),
        "experts' swiglu": lambda **s: nq.swiglu_fp8_experts(x, xs, w, ws, v, vs, ends, rows=rows, dtype=E4M3, **s),
        "route": lambda **s: nq.moe_route(logits, 4, **s),
        "combine": lambda **s: nq.moe_combine(a, slots, weights, **s),
        "sample": lambda **s: nq.sample(logits, noise, **s),
    }


def several(y):
    return y if isinstance(y, tuple) else (y,)


@pytest.mark.parametrize("name", ["quant", "gemm", "swiglu", "experts", "experts' swiglu", "route", "combine", "sample"])
def test_results_are_not_in_memory_that_the_current_stream_still_writes(name):
    call = calls(torch.Generator(device="cuda").manual_seed(3))[name]
    want = several(call())
    torch.cuda.synchronize()
    other, current = torch.cuda.Stream(), torch.cuda.current_stream()
    for _ in range(5):
        torch.cuda.empty_cache()
        junk = [torch.empty_like(y).view(torch.uint8) for y in want]
        places = {j.data_ptr() for j in junk}
        writes = torch.cuda.CUDAGraph()
        with torch.cuda.graph(writes):
            for _ in range(500):
                for j in junk:
                    j.fill_(255)
        writes.replay()                  # some milliseconds
        del junk, j                      # their memory is free for the current stream's next tensors
        got = several(call(stream=other))
        assert not places & {y.data_ptr() for y in got}
        current.wait_stream(other)
        read = [y.clone() for y in got]
        # freed while those copies wait: what the other stream does next leaves it alone
        del got
        junk = [y.view(torch.uint8) for y in several(call(stream=other))]
        with torch.cuda.stream(other):
            for j in junk:
                j.fill_(255)
        torch.cuda.synchronize()
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(read, want))
        del writes, junk, j


@pytest.mark.parametrize("name", ["quant", "gemm", "experts' swiglu", "route", "combine"])
def test_a_branch_of_a_captured_graph(name):
    call = calls(torch.Generator(device="cuda").manual_seed(4))[name]
    want = several(call())
    torch.cuda.synchronize()
    other, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        current = torch.cuda.current_stream()
        other.wait_stream(current)
        for _ in range(3):               # results made and dropped
            got = several(call(stream=other))
        current.wait_stream(other)
        read = [y.clone() for y in got]
        del got
        more = several(call())
    for _ in range(3):
        graph.replay()
        torch.cuda.synchronize()
        for y in (read, more):
            assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(y, want))
    again = several(call(stream=torch.cuda.default_stream()))
    torch.cuda.synchronize()
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(again, want))
