"""8-bit quantisation and products against plain forms in 64 bits, at the sizes, strides and groups where they can go
wrong. Tolerances: see fp8_ref."""
import pytest
import torch

from tests import fp8_ref as ref
from weight_only_groupwise_gb300 import nq

pytestmark = pytest.mark.gpu
BF16, FP16, F32, E4M3 = torch.bfloat16, torch.float16, torch.float32, ref.E4M3


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_only_groupwise_gb300 import build
    build.build()
    yield
    nq.device_error()


@pytest.fixture
def g(request):
    return torch.Generator(device="cuda").manual_seed(len(request.node.name))


def same(a, b):
    return torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# ---------------------------------------------------------------- quantisation

@pytest.mark.parametrize("dtype", [BF16, FP16, F32])
@pytest.mark.parametrize("rows,K", [(1, 16), (1, 128), (3, 144), (7, 1024), (65, 1040), (5, 5120), (2, 17408), (1000, 256)])
def test_quant(dtype, rows, K, g):
    x = (torch.randn((rows, K), device="cuda", generator=g) * torch.exp(2 * torch.randn((rows, 1), device="cuda", generator=g))).to(dtype)
    codes, scales = nq.quant_fp8(x)
    c, s = ref.quantised(x)
    assert torch.equal(scales, s) and same(codes.contiguous(), c.contiguous())


def test_quant_of_strided_rows_leaves_the_rest_alone(g):
    x = torch.randn((9, 640), device="cuda", generator=g).to(BF16)
    codes = torch.full((9, 400), 7, dtype=torch.uint8, device="cuda").view(E4M3)
    scales = torch.full((9, 11), -1.0, device="cuda")
    nq.quant_fp8(x[:, 128:400], out=(codes[:, 16:288], scales[:, 2:5]))
    c, s = ref.quantised(x[:, 128:400])
    assert torch.equal(scales[:, 2:5], s) and same(codes[:, 16:288].contiguous(), c.contiguous())
    left = codes.view(torch.uint8)
    assert bool((left[:, :16] == 7).all()) and bool((left[:, 288:] == 7).all())
    assert bool((scales[:, :2] == -1).all()) and bool((scales[:, 5:] == -1).all())


@pytest.mark.parametrize("dtype", [BF16, FP16, F32])
def test_quant_of_zeros_small_and_unusual_values(dtype):
    x = torch.zeros((6, 256), device="cuda", dtype=dtype)
    x[1, 5] = float("inf")
    x[2, 7] = float("nan")
    x[3] = torch.finfo(dtype).smallest_normal
    x[4, :128] = torch.finfo(dtype).max
    x[5, 3] = -0.0
    codes, scales = nq.quant_fp8(x)
    f = codes.float()
    floor = 2.0 ** -126
    assert bool((scales[0] == floor).all()) and bool((f[0] == 0).all())
    assert float(scales[1, 0]) == float("inf") and bool(f[1, 5].isnan()) and bool((f[1, 8:128] == 0).all())
    assert bool(scales[2, 0].isnan()) and bool(f[2, :128].isnan().all())
    assert float(scales[1, 1]) == float(scales[2, 1]) == floor and bool((f[1:3, 128:] == 0).all())
    want = max(torch.finfo(dtype).smallest_normal / 448, floor)
    assert bool((scales[3] == torch.tensor(want, device="cuda", dtype=F32)).all())
    assert bool((f[4, :128] == 448).all()) and bool((f[5] == 0).all())


# ---------------------------------------------------------------- dense products

SIZES = [(1, 16, 1), (1, 128, 128), (3, 144, 17), (8, 1040, 130), (16, 512, 1000), (17, 2048, 129), (33, 400, 515), (64, 1152, 384),
         (65, 96, 256), (127, 640, 200), (129, 384, 300), (200, 4096, 261), (300, 272, 1040), (513, 128, 64)]


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,K,N", SIZES)
def test_gemm(T, K, N, dtype, g):
    (x, xs), (w, ws) = ref.activations(T, K, g), ref.weights(1, N, K, g)
    xs = xs * 2.0 ** -12                 # within fp16's range
    y = nq.gemm_fp8(x, xs, w[0], ws[0], dtype=dtype)
    ref.close(y, *ref.product(x.double() * ref.spread(xs, K), ref.dense(w[0], ws[0])))


@pytest.mark.parametrize("dtype", [BF16, FP16, E4M3])
@pytest.mark.parametrize("T,K,N", [(1, 128, 16), (5, 400, 144), (16, 1024, 256), (40, 272, 400), (100, 144, 1040), (130, 640, 272), (300, 1040, 128)])
def test_swiglu(T, K, N, dtype, g):
    x, xs = ref.activations(T, K, g)
    w = [ref.weights(1, N, K, g) for _ in range(2)]
    xs = xs * 2.0 ** -9
    h = nq.swiglu_fp8(x, xs, w[0][0][0], w[0][1][0], w[1][0][0], w[1][1][0], dtype=dtype)
    a = x.double() * ref.spread(xs, K)
    want = ref.silu(*ref.product(a, ref.dense(w[0][0][0], w[0][1][0])), *ref.product(a, ref.dense(w[1][0][0], w[1][1][0])))
    ref.close_codes(*h, *want) if dtype is E4M3 else ref.close(h, *want)


def test_gemm_takes_any_strides(g):
    T, K, N = 37, 272, 150
    x, xs = ref.activations(T, K, g, stride=320)
    wide, ws = ref.weights(1, N, 400, g)
    w, ws = wide[0][:, 64:64 + K], ws[0][:, :3]
    xs = (torch.cat([xs, xs, xs], 1) * 2.0 ** -9)[:, 1:4]
    out = torch.full((T + 2, N + 7), 3.0, dtype=BF16, device="cuda")
    y = nq.gemm_fp8(x, xs, w, ws, out=out[1:T + 1, 3:3 + N])
    ref.close(y, *ref.product(x.double() * ref.spread(xs, K), ref.dense(w, ws)))
    out[1:T + 1, 3:3 + N] = 3.0
    assert bool((out == 3).all())


def test_a_nan_stays_in_its_row_and_column(g):
    T, K, N = 150, 256, 200
    (x, xs), (w, ws) = ref.activations(T, K, g), ref.weights(1, N, K, g)
    x.view(torch.uint8)[70, 40] = 0x7F
    w.view(torch.uint8)[0, 130, 200] = 0xFF
    y = nq.gemm_fp8(x, xs * 2.0 ** -9, w[0], ws[0])
    bad = torch.zeros((T, N), dtype=torch.bool, device="cuda")
    bad[70] = True
    bad[:, 130] = True
    assert torch.equal(y.isnan(), bad)
    # an infinite scale too
    xs[3, 1] = float("inf")
    assert not bool(nq.gemm_fp8(x, xs * 2.0 ** -9, w[0], ws[0])[3].isfinite().any())


def test_sums_that_cancel(g):
    """Blocks whose sums are large and cancel leave what 32-bit sums leave."""
    T, K, N = 20, 2048, 128
    (x, xs), (w, ws) = ref.activations(T, K // 2, g), ref.weights(1, N, K // 2, g)
    x, xs = torch.cat([x, x], 1), torch.cat([xs, xs], 1) * 2.0 ** -9
    w, ws = torch.cat([w[0].float(), -w[0].float()], 1).to(E4M3), torch.cat([ws[0], ws[0]], 1)
    y = nq.gemm_fp8(x, xs, w, ws)
    ref.close(y, *ref.product(x.double() * ref.spread(xs, K), ref.dense(w, ws)))


def test_the_same_call_twice_gives_the_same_bits(g):
    for T, K, N in ((5, 5120, 1000), (200, 2048, 640)):
        (x, xs), (w, ws) = ref.activations(T, K, g), ref.weights(1, N, K, g)
        a = nq.gemm_fp8(x, xs, w[0], ws[0])
        assert all(same(a, nq.gemm_fp8(x, xs, w[0], ws[0])) for _ in range(3))


# ---------------------------------------------------------------- experts

def check_experts(x, xs, w, offsets, rows, dtype, out=None):
    E, N, K = w[0][0].shape
    ends = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    call = nq.gemm_fp8_experts if len(w) == 1 else nq.swiglu_fp8_experts
    y = call(x, xs, *[t for pair in w for t in pair], ends, rows=rows, dtype=dtype, out=out)
    a = x.double() * ref.spread(xs, K)
    if rows is not None:
        there = (rows >= 0) & (rows < x.shape[0])
        a = torch.where(there[:, None], a[rows.clamp(0, x.shape[0] - 1).long()], 0.0)
    for e in range(E):
        r0, r1 = offsets[e], offsets[e + 1]
        if r0 == r1:
            continue
        parts = [ref.product(a[r0:r1], ref.dense(c[e], s[e])) for c, s in w]
        want = parts[0] if len(w) == 1 else ref.silu(*parts[0], *parts[1])
        if dtype is E4M3:
            ref.close_codes(y[0][r0:r1], y[1][r0:r1], *want)
        else:
            ref.close(y[r0:r1], *want)
    return y


GROUPS = [[0, 0, 5, 5, 6, 40], [0, 130, 131, 131, 300], [0, 1, 2, 3, 4, 5, 6, 7, 8], [0, 0, 0, 0], [0, 64, 128, 384, 390], [0, 700]]


@pytest.mark.parametrize("gather", [False, True])
@pytest.mark.parametrize("dtype,glu", [(BF16, False), (FP16, False), (BF16, True), (E4M3, True)])
@pytest.mark.parametrize("offsets", GROUPS, ids=str)
def test_experts(offsets, dtype, glu, gather, g):
    E, M, K, N = len(offsets) - 1, offsets[-1], 400, 272
    x, xs = ref.activations(max(M // 3, 2) if gather else max(M, 1), K, g)
    rows = torch.randint(0, x.shape[0], (M,), device="cuda", generator=g, dtype=torch.int32) if gather else None
    w = [ref.weights(E, N, K, g) for _ in range(1 + glu)]
    check_experts(x, xs * 2.0 ** -10, w, offsets, rows, dtype)


@pytest.mark.parametrize("glu", [False, True])
@pytest.mark.parametrize("E,M,K,N", [(130, 200, 128, 64), (8, 1000, 1040, 515), (3, 2000, 256, 1), (512, 90, 64, 48), (16, 17, 2048, 768)])
def test_many_and_uneven_experts(E, M, K, N, glu, g):
    if glu:
        N = -(-N // 16) * 16
    cuts = torch.randint(0, M + 1, (E - 1,), device="cuda", generator=g).sort().values.tolist()
    x, xs = ref.activations(M, K, g)
    rows = torch.randperm(M, device="cuda", generator=g).to(torch.int32)
    check_experts(x, xs * 2.0 ** -10, [ref.weights(E, N, K, g) for _ in range(1 + glu)], [0, *cuts, M], rows, E4M3 if glu else BF16)


def test_rows_outside_x_read_as_zeros_and_rows_of_no_expert_are_left(g):
    K, N = 272, 140
    x, xs = ref.activations(10, K, g)
    xs[0] = float("nan")                 # a row that nothing takes
    rows = torch.randint(1, 10, (300,), device="cuda", generator=g, dtype=torch.int32)
    rows[::7] = torch.tensor([-1, 10, 1 << 30, -(1 << 31)], device="cuda", dtype=torch.int32).repeat(11)[:43]
    out = torch.full((300, N), 5.0, dtype=BF16, device="cuda")
    y = check_experts(x, xs * 2.0 ** -9, [ref.weights(3, N, K, g)], [20, 100, 100, 260], rows, BF16, out=out)
    assert bool((y[:20] == 5).all()) and bool((y[260:] == 5).all()) and bool((y[20:260][(rows[20:260] < 0) | (rows[20:260] > 9)] == 0).all())


def test_offsets_are_clamped(g):
    K, N, M = 128, 128, 50
    x, xs = ref.activations(M, K, g)
    w, ws = ref.weights(3, N, K, g)
    ends = torch.tensor([-7, 20, 10, 1 << 30], dtype=torch.int32, device="cuda")
    y = nq.gemm_fp8_experts(x, xs, w, ws, ends)
    # 0..20 are the first expert's, none the second's, 10.. the third's, which wins or loses 10..20
    a = x.double() * ref.spread(xs, K)
    ref.close(y[:10], *ref.product(a[:10], ref.dense(w[0], ws[0])))
    ref.close(y[20:], *ref.product(a[20:], ref.dense(w[2], ws[2])))


def test_gate_and_up_as_halves_of_one_tensor_and_every_other_expert(g):
    E, K, N = 3, 256, 128
    c, s = ref.weights(2 * E, 2 * N, K, g)
    x, xs = ref.activations(90, K, g)
    w = [(c[::2, :N], s[::2, :1]), (c[::2, N:], s[::2, 1:])]
    check_experts(x, xs * 2.0 ** -9, w, [0, 30, 31, 90], None, BF16)


# ---------------------------------------------------------------- streams and graphs

def test_on_another_stream_and_in_graphs_that_run_at_once(g):
    K, N = 512, 384
    sets = [(ref.activations(T, K, g), ref.weights(1, N, K, g)) for T in (3, 150, 40)]
    want = [nq.gemm_fp8(x, xs, w[0], ws[0]) for (x, xs), (w, ws) in sets]
    outs, graphs, streams = [], [], [torch.cuda.Stream() for _ in sets]
    for ((x, xs), (w, ws)), stream in zip(sets, streams):
        out = torch.empty((x.shape[0], N), dtype=BF16, device="cuda")
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(4):
                nq.gemm_fp8(x, xs, w[0], ws[0], out=out)
        outs.append(out)
        graphs.append(graph)
    for _ in range(3):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for graph, stream in zip(graphs, streams):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        assert all(same(a, b) for a, b in zip(outs, want))
    with torch.cuda.stream(streams[0]):
        again = nq.gemm_fp8(*sets[1][0], sets[1][1][0][0], sets[1][1][1][0])
    torch.cuda.synchronize()
    assert same(again, want[1])


def test_empty_calls(g):
    x, xs = ref.activations(1, 128, g)
    w, ws = ref.weights(2, 64, 128, g)
    assert nq.gemm_fp8(x[:0], xs[:0], w[0], ws[0]).shape == (0, 64)
    none = torch.zeros(3, dtype=torch.int32, device="cuda")
    assert nq.gemm_fp8_experts(x[:0], xs[:0], w, ws, none).shape == (0, 64)
    assert nq.quant_fp8(torch.empty((0, 128), device="cuda"))[0].shape == (0, 128)
    # rows that all lie outside an empty x
    rows = torch.zeros(5, dtype=torch.int32, device="cuda")
    ends = torch.tensor([0, 2, 5], dtype=torch.int32, device="cuda")
    assert bool((nq.gemm_fp8_experts(x[:0], xs[:0], w, ws, ends, rows=rows) == 0).all())


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("E,M,K,N", [(8, 200, 1040, 515), (16, 331, 256, 144), (40, 1280, 640, 272), (3, 96, 144, 1)])
def test_sorted_rows_of_some_tens_an_expert(E, M, K, N, dtype, g):
    """One expert has none, one two thirds of the rows."""
    cuts = sorted(torch.randint(0, M // 3 + 1, (E - 2,), device="cuda", generator=g).tolist())
    x, xs = ref.activations(M, K, g)
    check_experts(x, xs * 2.0 ** -10, [ref.weights(E, N, K, g)], [0, 0, *cuts, M], None, dtype)


@pytest.mark.parametrize("E,M,K,N", [(8, 200, 1040, 515), (16, 331, 256, 144), (3, 96, 144, 1)])
def test_gathered_rows_of_some_tens_an_expert(E, M, K, N, g):
    """Copied together first; rows that x has not are zeros."""
    cuts = sorted(torch.randint(0, M // 3 + 1, (E - 2,), device="cuda", generator=g).tolist())
    x, xs = ref.activations(50, K, g)
    rows = torch.randint(-1, 52, (M,), device="cuda", generator=g, dtype=torch.int32)
    check_experts(x, xs * 2.0 ** -10, [ref.weights(E, N, K, g)], [0, 0, *cuts, M], rows, BF16)


@pytest.mark.parametrize("dtype,glu", [(BF16, False), (E4M3, True)])
@pytest.mark.parametrize("E,M,K,N", [(8, 200, 1040, 512), (2, 700, 256, 272), (1, 130, 144, 48)])
def test_gathered_rows_without_scratch_memory(E, M, K, N, dtype, glu, g, monkeypatch):
    monkeypatch.setattr(nq.lib(), "nq_fp8_scratch_bytes", lambda *a: 0)
    x, xs = ref.activations(50, K, g)
    rows = torch.randint(-1, 52, (M,), device="cuda", generator=g, dtype=torch.int32)
    cuts = sorted(torch.randint(0, M + 1, (E - 1,), device="cuda", generator=g).tolist())
    check_experts(x, xs * 2.0 ** -10, [ref.weights(E, N, K, g) for _ in range(1 + glu)], [0, *cuts, M], rows, dtype)
