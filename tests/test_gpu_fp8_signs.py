"""Signs of quantised values: of zeros too, and of what is rounded to zero."""
import pytest
import torch

from tests import fp8_ref as ref
from weight_only_groupwise_gb300 import nq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_only_groupwise_gb300 import build
    build.build()
    yield
    nq.device_error()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16, torch.float32])
@pytest.mark.parametrize("size", [1.0, 2.0 ** -13, 2.0 ** 13, 2.0 ** -70, 2.0 ** 70])
def test_signs_are_kept(dtype, size):
    """Blocks whose scales are near one, far from it, and out of the range of the corrected quotients."""
    if not torch.finfo(dtype).smallest_normal <= size <= torch.finfo(dtype).max / 4:
        pytest.skip("not in the type's range")
    g = torch.Generator(device="cuda").manual_seed(int(torch.tensor(size).log2()) + 100)
    x = (torch.randn((50, 400), device="cuda", generator=g) * size).to(dtype)
    x[:, ::5] = 0.0
    x[:, 1::5] = -0.0
    x[:, 2::15] *= 2.0 ** -12            # codes of zero, with a sign
    x[3] = 0.0
    x[4] = -0.0
    codes, scales = nq.quant_fp8(x)
    want, s = ref.quantised(x)
    assert torch.equal(scales, s)
    assert torch.equal(codes.view(torch.uint8), want.contiguous().view(torch.uint8))
    assert torch.equal(codes.float().signbit(), x.signbit())


def test_every_code(dtype=torch.float32):
    """All values of a block of scale 1, and what lies halfway between neighbours and next to that."""
    v = torch.arange(256, device="cuda", dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).float()
    v = v[v.isfinite()]
    up = v.sort().values
    mid = (up[1:] + up[:-1]) / 2
    inf = torch.tensor(float("inf"), device="cuda")
    v = torch.cat([v, mid, torch.nextafter(mid, inf), torch.nextafter(mid, -inf)])
    v = torch.nn.functional.pad(v, (0, -len(v) % 127))
    x = torch.nn.functional.pad(v.view(-1, 127), (0, 1), value=448.0).contiguous()
    for x in (x, -x, x * 2.0 ** -20):
        codes, scales = nq.quant_fp8(x)
        want, s = ref.quantised(x)
        assert torch.equal(scales, s) and torch.equal(codes.view(torch.uint8), want.contiguous().view(torch.uint8))
