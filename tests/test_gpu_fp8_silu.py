"""SwiGLU results over the whole range of the gate, where its exponential leaves fp32's normal numbers among it."""
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


def gates(T):
    """T gates: all of -104 to -80, and the rest of the range."""
    few = torch.tensor([-87.34, -88.0, -88.7, -88.73, -100.0, -1e30, 1e30, 0.0, 88.0, 100.0, -1.0, 1.0, -20.0, 20.0, -87.0, -86.0], device="cuda")
    return torch.cat([few, torch.linspace(-104, -80, 2048, device="cuda")[::2048 // T]])[:T].contiguous()


# rows a call: 16 and 32 in tiles of the kernel for few rows, dense calls with their sums shared by a cluster, the kernel for many
@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,K,dense", [(16, 256, False), (28, 256, False), (600, 256, False), (16, 2048, True), (50, 2048, True), (64, 128, True),
                                       (2000, 128, True)])
def test_silu_of_far_gates(T, K, dense, dtype):
    """A gate is its row's scale (codes 1 and 0), u the same times a power of two that brings their product into the result's range."""
    N, g = 48, gates(T)
    x = torch.zeros((T, K), device="cuda")
    x[:, K // 2] = 1
    wg = torch.zeros((N, K), device="cuda")
    wg[:, K // 2] = 1
    wu = wg * torch.where(torch.arange(N, device="cuda") % 3 == 0, -0.5, 1.5)[:, None]
    xs = g[:, None].expand(T, K // 128).contiguous()
    ones = torch.ones((1, K // 128), device="cuda")
    x, wg, wu, su = x.to(E4M3), wg.to(E4M3), wu.to(E4M3), ones * 2.0 ** 110
    if dense:
        h = nq.swiglu_fp8(x, xs, wg, ones, wu, su, dtype=dtype)
    else:
        ends = torch.tensor([0, T], dtype=torch.int32, device="cuda")
        h = nq.swiglu_fp8_experts(x, xs, wg[None], ones[None], wu[None], su[None], ends, dtype=dtype)
    gd = g.double()[:, None]
    u = gd * su[0, 0].double() * wu[:, K // 2].double()
    want = gd * torch.where(gd < 0, torch.exp(gd.clamp(max=0)), 1.0) / (1 + torch.exp(-gd.abs())) * u
    # the exponential: 2 + 1.173 |g| last places (as CUDA documents it; 2^-149 at least), the quotient two, u, a sum and two
    # products a half each
    err = (6 + 1.173 * gd.abs().clamp(max=200)) * 2.0 ** -23 * want.abs() + (gd * u).abs() * 2.0 ** -148 * (gd > -1000)
    fits = (u.abs() < 2.0 ** 127) & (want.abs() + err < torch.finfo(dtype).max)
    assert int(fits.sum()) > T * N // 4
    bad = ~fits
    ref.close(torch.where(bad, 0.0, h), torch.where(bad, 0.0, want), torch.where(bad, 0.0, err))
