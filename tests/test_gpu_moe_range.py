"""The router's weights over the whole range of scores, chosen ones far apart among them."""
import pytest
import torch

from weight_only_groupwise_gb300 import nq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_only_groupwise_gb300 import build
    build.build()
    yield
    nq.device_error()


def rows(T):
    """Logits [T][16] of which four are chosen (all others are 16 lower than those, or masked): from well above zero to where a
    score has no place in 32 bits."""
    g = torch.Generator(device="cuda").manual_seed(T)
    x = torch.full((T, 16), -float("inf"), device="cuda")
    x[:, :4] = torch.empty((T, 4), device="cuda").uniform_(-130, 20, generator=g)
    x[:T // 3, :4] = torch.empty((T // 3, 4), device="cuda").uniform_(-100, -30, generator=g)
    x[0, :4] = torch.tensor([-59.0, -89.0, -59.5, -88.0])
    x[1, :4] = torch.tensor([-39.0, -89.0, -120.0, -40.0])
    x[2, :4] = torch.tensor([-50.0, -100.0, -61.0, -103.0])
    x[3, :4] = torch.tensor([-60.0, -60.5, -90.0, -140.0])
    x[4, :4] = torch.tensor([0.0, -0.0, -86.0, -87.5])
    x[5, :4] = torch.tensor([float("inf"), 3.0, -80.0, -100.0])
    x[6, :4] = torch.tensor([-1e30, -1e30, -2e30, -3e38])
    x[7, :4] = torch.tensor([30.0, 90.0, -85.0, 0.5])
    return x


@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("normalize", [True, False])
@pytest.mark.parametrize("T", [40, 700])
def test_sigmoid_weights(T, normalize, biased):
    x = rows(T)
    bias = torch.zeros(16, device="cuda") if biased else None
    ids, w, *_ = nq.moe_route(x, 4, score="sigmoid", normalize=normalize, scale=2.5, bias=bias)
    assert torch.equal(ids.sort(1).values, torch.arange(4, device="cuda", dtype=torch.int32).expand(T, 4))
    c = x.double().gather(1, ids.long())
    log = torch.nn.functional.logsigmoid(c)
    if normalize:
        far = log.amax(1, keepdim=True)
        want = torch.exp(log - far)
        want = 2.5 * want / want.sum(1, keepdim=True)
        # what the exponentials are taken of is a difference of logits, rounded (2^-24 of it)
        most = (c - c.amax(1, keepdim=True).clamp(max=0)).clamp(min=-200, max=0).abs()
    else:
        want = 2.5 * torch.exp(log)
        most = torch.zeros_like(c)
    # and half places (2^-24): a score's two exponentials four each, 1 + e and the quotient one each, ten together; their sum the
    # same, its five rounds of additions, and less than |d| e^-|d| < 1/2 for each rounded difference d; a quotient and the scale
    # two: fewer than 32. Numbers below the smallest normal one (2^-126) lose places.
    bound = (most + 32) * 2.0 ** -24 * want + 4 * 2.0 ** -126
    assert bool(((w.double() - want).abs() <= bound).all())
