"""8-bit products of many rows at the sizes of a prompt's layers: sums of more blocks of K than go by bulk copies, with results
aligned to 16 bytes, whose tiles leave as whole lines; sums that cancel. Tolerances: see fp8_ref."""
import pytest
import torch

from tests import fp8_ref as ref
from weight_only_groupwise_gb300 import nq

pytestmark = pytest.mark.gpu
BF16, FP16, E4M3 = torch.bfloat16, torch.float16, ref.E4M3


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_only_groupwise_gb300 import build
    build.build()
    yield
    nq.device_error()


@pytest.fixture
def g(request):
    return torch.Generator(device="cuda").manual_seed(len(request.node.name))


# 27B-class projections of a prompt's rows, the last tile of rows and of columns not full; N of no whole 128, of no whole 16
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,K,N", [(2000, 4240, 2040), (1200, 5120, 2056), (513, 17408, 5120), (700, 5120, 17408), (1025, 6144, 2504)])
def test_gemm_of_long_sums(T, K, N, dtype, g):
    (x, xs), (w, ws) = ref.activations(T, K, g), ref.weights(1, N, K, g)
    xs = xs * 2.0 ** -12
    y = nq.gemm_fp8(x, xs, w[0], ws[0], dtype=dtype)
    ref.close(y, *ref.product(x.double() * ref.spread(xs, K), ref.dense(w[0], ws[0])))


@pytest.mark.parametrize("T,K,N", [(700, 5120, 1032), (300, 4224, 264), (129, 8192, 8), (2000, 4240, 520)])
def test_one_experts_rows(T, K, N, g):
    """The same kernel at sizes for which a dense call takes another; columns between results are left alone."""
    (x, xs), (w, ws) = ref.activations(T, K, g), ref.weights(1, N, K, g)
    xs = xs * 2.0 ** -12
    out = torch.full((T + 1, N + 16), 3.0, device="cuda", dtype=BF16)
    y = nq.gemm_fp8_experts(x, xs, w, ws, torch.tensor([0, T], dtype=torch.int32, device="cuda"), out=out[:T, 8:8 + N])
    ref.close(y, *ref.product(x.double() * ref.spread(xs, K), ref.dense(w[0], ws[0])))
    y.fill_(3.0)
    assert bool((out == 3).all())


@pytest.mark.parametrize("dtype", [BF16, E4M3])
@pytest.mark.parametrize("T,K,N", [(1300, 4240, 1040), (600, 5120, 4112)])
def test_swiglu_of_long_sums(T, K, N, dtype, g):
    x, xs = ref.activations(T, K, g)
    w = [ref.weights(1, N, K, g) for _ in range(2)]
    xs = xs * 2.0 ** -10
    h = nq.swiglu_fp8(x, xs, w[0][0][0], w[0][1][0], w[1][0][0], w[1][1][0], dtype=dtype)
    a = x.double() * ref.spread(xs, K)
    want = ref.silu(*ref.product(a, ref.dense(w[0][0][0], w[0][1][0])), *ref.product(a, ref.dense(w[1][0][0], w[1][1][0])))
    ref.close_codes(*h, *want) if dtype is E4M3 else ref.close(h, *want)


@pytest.mark.parametrize("T,K,N", [(1200, 2048, 2056), (1200, 8448, 2056), (200, 4096, 520)])
def test_sums_that_cancel(T, K, N, g):
    """Blocks whose sums are large and cancel leave what 32-bit sums leave."""
    (x, xs), (w, ws) = ref.activations(T, K // 2, g), ref.weights(1, N, K // 2, g)
    x, xs = torch.cat([x, x], 1), torch.cat([xs, xs], 1) * 2.0 ** -9
    w, ws = torch.cat([w[0].float(), -w[0].float()], 1).to(E4M3), torch.cat([ws[0], ws[0]], 1)
    ref.close(nq.gemm_fp8(x, xs, w, ws), *ref.product(x.double() * ref.spread(xs, K), ref.dense(w, ws)))
