"""8-bit products and experts at the edges of what is allowed: waits that run out, the first call of a process inside a
capture, other streams, weights that experts share, tensors past 2^32 elements, calls that follow each other closely."""
import os
import subprocess
import sys

import pytest
import torch

from tests import fp8_ref as ref
from tests.gpu_util import expect_timeout
from weight_only_groupwise_gb300 import nq

pytestmark = pytest.mark.gpu
BF16, E4M3 = torch.bfloat16, ref.E4M3
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_only_groupwise_gb300 import build
    build.build()
    yield
    nq.device_error()


@pytest.fixture
def g():
    return torch.Generator(device="cuda").manual_seed(7)


def same(a, b):
    return torch.equal(a.contiguous().view(torch.uint8), b.contiguous().view(torch.uint8))


def experts_call(E, M, K, N, glu, gather, g, **how):
    x, xs = ref.activations(M, K, g)
    w = [ref.weights(E, N, K, g) for _ in range(1 + glu)]
    cuts = torch.randint(0, M + 1, (E - 1,), device="cuda", generator=g).sort().values.to(torch.int32)
    ends = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), M)])
    rows = torch.randperm(M, device="cuda", generator=g).to(torch.int32) if gather else None
    fn = nq.swiglu_fp8_experts if glu else nq.gemm_fp8_experts
    return lambda **more: fn(x, xs * 2.0 ** -10, *[t for p in w for t in p], ends, rows=rows, **how, **more)


def dense_call(T, K, N, glu, g, **how):
    x, xs = ref.activations(T, K, g)
    w = [ref.weights(1, N, K, g) for _ in range(1 + glu)]
    fn = nq.swiglu_fp8 if glu else nq.gemm_fp8
    return lambda **more: fn(x, xs * 2.0 ** -10, *[t for c, s in w for t in (c[0], s[0])], **how, **more)


CALLS = {
    "one block a tile": lambda g: dense_call(16, 2048, 17408, False, g),
    "split": lambda g: dense_call(40, 5120, 1024, False, g),
    "split swiglu": lambda g: dense_call(30, 4096, 1024, True, g, dtype=E4M3),
    "many rows": lambda g: dense_call(2000, 4096, 2048, False, g),
    "many rows, short sums": lambda g: dense_call(2000, 1024, 2048, False, g),
    "many rows, swiglu": lambda g: dense_call(1500, 2048, 1024, True, g, dtype=E4M3),
    "experts": lambda g: experts_call(64, 200, 2048, 512, True, True, g, dtype=E4M3),
    "experts, many rows": lambda g: experts_call(4, 1500, 2048, 512, False, True, g),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(name, g):
    call = CALLS[name](g)
    first = call()
    nq.device_error()
    expect_timeout(nq, call)
    for a, b in zip(*[r if isinstance(r, tuple) else (r,) for r in (first, call())]):
        assert same(a, b)
    nq.device_error()


@pytest.mark.parametrize("name", CALLS)
def test_calls_behind_each_other_with_changing_inputs(name, g):
    """Many calls without a wait between, each with inputs that a kernel just before has written."""
    call = CALLS[name](g)
    x = [c.cell_contents for c in call.__closure__ if isinstance(c.cell_contents, torch.Tensor) and c.cell_contents.dtype is E4M3][0]
    bytes_ = x.view(torch.uint8)
    inputs = [bytes_.roll(i, 1).clone() for i in range(3)]
    want = []
    for i in inputs:
        bytes_.copy_(i)
        torch.cuda.synchronize()
        want.append(call())
        torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for i in inputs:
            bytes_.copy_(i)
            got.append(call())
        for a, b in zip(got, want):
            for p, q in zip(*[r if isinstance(r, tuple) else (r,) for r in (a, b)]):
                assert same(p, q)


def test_quantised_rows_straight_into_a_product(g):
    (w, ws) = ref.weights(1, 640, 1024, g)
    xs = [torch.randn((70, 1024), device="cuda", generator=g).to(BF16) for _ in range(4)]
    want = []
    for x in xs:
        q = nq.quant_fp8(x)
        torch.cuda.synchronize()
        want.append(nq.gemm_fp8(*q, w[0], ws[0]))
        torch.cuda.synchronize()
    out = nq.quant_fp8(xs[0])
    for _ in range(20):
        got = [nq.gemm_fp8(*nq.quant_fp8(x, out=out), w[0], ws[0]) for x in xs]
        assert all(same(a, b) for a, b in zip(got, want))


def test_weights_quantised_just_before(g):
    """nq_quant_fp8's codes as a weight (one block of 128 rows, one scale each 128 x 128 put in by hand)."""
    x, xs = ref.activations(16, 512, g)
    ws = torch.ones((1, 4), device="cuda")
    w = [torch.randn((128, 512), device="cuda", generator=g).to(BF16) for _ in range(2)]
    want = [nq.gemm_fp8(x, xs, nq.quant_fp8(v)[0].clone(), ws) for v in w]
    torch.cuda.synchronize()
    out = nq.quant_fp8(w[0])
    for _ in range(20):
        for v, y in zip(w, want):
            assert same(nq.gemm_fp8(x, xs, nq.quant_fp8(v, out=out)[0], ws), y)


@pytest.mark.parametrize("T", [48, 600])
def test_weights_that_a_swiglu_has_just_written(T, g):
    """nq_swiglu_fp8's codes as a weight, from either kernel."""
    K, N = 1024, 512
    x, xs = ref.activations(16, N, g)
    a = [ref.activations(T, K, g) for _ in range(2)]
    (wg, sg), (wu, su) = ref.weights(1, N, K, g), ref.weights(1, N, K, g)
    ws = torch.ones((-(-T // 128), N // 128), device="cuda")
    codes = lambda i, out=None: nq.swiglu_fp8(*a[i], wg[0], sg[0], wu[0], su[0], dtype=torch.float8_e4m3fn, out=out)  # noqa: E731
    want = []
    for i in range(2):
        w = codes(i)[0].clone()
        torch.cuda.synchronize()
        want.append(nq.gemm_fp8(x, xs, w, ws))
        torch.cuda.synchronize()
    assert not same(*want)
    out, got = codes(0), [torch.empty_like(y) for y in want]
    graph = torch.cuda.CUDAGraph()           # kernels close behind each other
    with torch.cuda.graph(graph):
        for i in range(2):
            nq.gemm_fp8(x, xs, codes(i, out)[0], ws, out=got[i])
    for _ in range(20):
        graph.replay()
        assert all(same(a, b) for a, b in zip(got, want))


def test_on_a_stream_that_is_not_the_current_one(g):
    call = CALLS["experts, many rows"](g)
    want = call()
    torch.cuda.synchronize()
    other = torch.cuda.Stream()
    for _ in range(5):
        out = torch.empty_like(want)
        torch.cuda.synchronize()
        call(out=out, stream=other)
        junk = [torch.full((1500 * 2100,), 255, dtype=torch.uint8, device="cuda") for _ in range(3)]  # what scratch was
        other.synchronize()
        assert same(out, want)
        del junk


def test_on_a_stream_while_the_current_one_still_writes_freed_memory(g):
    call = CALLS["experts, many rows"](g)
    want = call()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    other, need = torch.cuda.Stream(), nq.lib().nq_fp8_scratch_bytes(1500, 4, 2048, 0)
    for _ in range(5):
        out = torch.empty_like(want)
        junk = torch.empty(need, dtype=torch.uint8, device="cuda")
        writes = torch.cuda.CUDAGraph()
        with torch.cuda.graph(writes):
            for _ in range(2000):
                junk.fill_(255)
        writes.replay()                      # some milliseconds
        del junk                             # its memory is free for the current stream's next tensors
        call(out=out, stream=other)
        torch.cuda.synchronize()
        assert same(out, want)
        del writes


def test_on_two_streams_at_once(g):
    """All kinds of calls on one stream in order, and in the opposite order on another, many of them in flight."""
    calls = [make(g) for make in CALLS.values()]
    flat = lambda y: y if isinstance(y, torch.Tensor) else y[0]  # noqa: E731
    want = [flat(call()).clone() for call in calls]
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(2)], [[], []]
    for _ in range(5):
        for s, order in ((0, 1), (1, -1)):
            with torch.cuda.stream(streams[s]):
                got[s] += [flat(call()) for call in calls[::order]]
    torch.cuda.synchronize()
    nq.device_error()
    for s, order in ((0, 1), (1, -1)):
        assert all(same(y, want[::order][i % len(calls)]) for i, y in enumerate(got[s]))


def test_experts_that_share_a_weight(g):
    (w, ws), (x, xs) = ref.weights(1, 200, 256, g), ref.activations(30, 256, g)
    ends = torch.tensor([0, 4, 4, 30], dtype=torch.int32, device="cuda")
    y = nq.gemm_fp8_experts(x, xs, w.expand(3, -1, -1), ws.expand(3, -1, -1), ends)
    assert same(y, nq.gemm_fp8_experts(x, xs, w.repeat(3, 1, 1), ws.repeat(3, 1, 1), ends))


def test_rows_past_2_to_the_32(g):
    T, K, N = 262500, 16384, 40
    x = torch.zeros((T, K), dtype=torch.uint8, device="cuda").view(E4M3)
    xs = torch.zeros((T, K // 128), device="cuda")
    few, scales = ref.activations(300, K, g)
    x.view(torch.uint8)[-300:] = few.view(torch.uint8)
    xs[-300:] = scales
    w, ws = ref.weights(1, N, K, g)
    want = nq.gemm_fp8(few, scales, w[0], ws[0])
    got = nq.gemm_fp8(x, xs, w[0], ws[0])
    a, err = ref.product(few.double() * ref.spread(scales, K), ref.dense(w[0], ws[0]))
    ref.close(got[-300:], a, err)
    ref.close(want, a, err)
    assert bool((got[:-300] == 0).all())
    rows = torch.arange(T - 1, T - 301, -1, device="cuda", dtype=torch.int32)
    for n in (300, 9):                   # copied together first, and gathered
        ends = torch.tensor([0, n], dtype=torch.int32, device="cuda")
        ref.close(nq.gemm_fp8_experts(x, xs, w, ws, ends, rows=rows[:n]), a.flip(0)[:n], err.flip(0)[:n])


def test_weights_past_2_to_the_32(g):
    E, N, K = 300, 1792, 8192
    w = torch.zeros((E, N, K), dtype=torch.uint8, device="cuda").view(E4M3)
    ws = torch.ones((E, N // 128, K // 128), device="cuda")
    last, _ = ref.activations(N, K, g)
    w.view(torch.uint8)[-1] = last.view(torch.uint8)
    x, xs = ref.activations(5, K, g)
    xs = xs * 2.0 ** -9
    ends = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    ends[-2:] = torch.tensor([1, 5])
    y = nq.gemm_fp8_experts(x, xs, w, ws, ends)
    ref.close(y[1:], *ref.product((x.double() * ref.spread(xs, K))[1:], ref.dense(last, ws[0])))
    assert bool((y[0] == 0).all())


FIRST = """
import sys, torch
sys.path.insert(0, {root!r})
from tests import fp8_ref as ref
from weight_only_groupwise_gb300 import nq
g = torch.Generator(device="cuda").manual_seed(1)
x, xs = ref.activations({T}, 512, g)
w, ws = ref.weights(2, 256, 512, g)
ends = torch.tensor([0, {T} // 2, {T}], dtype=torch.int32, device="cuda")
rows = torch.arange({T}, dtype=torch.int32, device="cuda").flip(0).contiguous()
logits = torch.randn(({T}, 40), device="cuda", generator=g)
torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y = nq.gemm_fp8(x, xs, w[0], ws[0])
    h = nq.swiglu_fp8_experts(x, xs, w, ws, w, ws, ends, rows=rows, dtype=ref.E4M3)
    r = nq.moe_route(logits, 4)
for _ in range(2):
    graph.replay()
torch.cuda.synchronize()
nq.device_error()
assert torch.equal(y, nq.gemm_fp8(x, xs, w[0], ws[0]))
assert all(torch.equal(a, b) for a, b in zip(r, nq.moe_route(logits, 4)))
again = nq.swiglu_fp8_experts(x, xs, w, ws, w, ws, ends, rows=rows, dtype=ref.E4M3)
assert torch.equal(h[0].view(torch.uint8), again[0].view(torch.uint8)) and torch.equal(h[1], again[1])
print("fine")
"""


@pytest.mark.parametrize("T", [6, 5000])
def test_the_first_call_of_a_process_inside_a_capture(T):
    r = subprocess.run([sys.executable, "-c", FIRST.format(root=ROOT, T=T)], capture_output=True, text=True, timeout=300, cwd=ROOT)
    assert r.returncode == 0 and "fine" in r.stdout, r.stderr[-2000:]
