"""8-bit products whose waits run out, with others right behind them. What an aborted block has asked for arrives before it
leaves, so that the next block on its SM finds its shared memory to itself."""
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


@pytest.fixture
def g():
    return torch.Generator(device="cuda").manual_seed(11)


def same(a, b):
    return all(torch.equal(p.view(torch.uint8), q.view(torch.uint8)) for p, q in zip(*[r if isinstance(r, tuple) else (r,) for r in (a, b)]))


def dense(T, K, N, glu, g, **how):
    x, xs = ref.activations(T, K, g)
    xs *= 2.0 ** -10                     # (here, so that no other kernel runs ahead of the call's)
    w = [ref.weights(1, N, K, g) for _ in range(1 + glu)]
    fn = nq.swiglu_fp8 if glu else nq.gemm_fp8
    return lambda: fn(x, xs, *[t for c, s in w for t in (c[0], s[0])], **how)


def experts(E, M, K, N, glu, g, **how):
    x, xs = ref.activations(M, K, g)
    xs *= 2.0 ** -10
    w = [ref.weights(E, N, K, g) for _ in range(1 + glu)]
    ends = torch.linspace(0, M, E + 1, device="cuda").to(torch.int32)
    rows = torch.randperm(M, device="cuda", generator=g).to(torch.int32)
    fn = nq.swiglu_fp8_experts if glu else nq.gemm_fp8_experts
    return lambda: fn(x, xs, *[t for p in w for t in p], ends, rows=rows, **how)


def limited(ns, call):
    """The call with waits of at most `ns`."""
    before = nq.wait_limit(ns)
    try:
        return call()
    finally:
        nq.wait_limit(before)


# all of a block's copies are asked for at once (K of no more blocks than stages, a few blocks a rank of a split sum), and not
CALLS = {
    "few rows, short": lambda g: dense(16, 512, 4096, False, g),
    "split": lambda g: dense(40, 5120, 1024, False, g),
    "split swiglu": lambda g: dense(30, 4096, 1024, True, g, dtype=E4M3),
    "many rows, short": lambda g: dense(2000, 384, 2048, False, g),
    "many rows, short swiglu": lambda g: dense(2000, 512, 1024, True, g, dtype=E4M3),
    "many rows, long": lambda g: dense(1200, 4240, 2048, False, g),
    "experts, gathered": lambda g: experts(40, 200, 384, 512, True, g, dtype=E4M3),
    "experts, many rows": lambda g: experts(4, 1500, 256, 512, False, g),
}


@pytest.mark.parametrize("name", CALLS)
def test_a_call_right_behind_one_that_gave_up_is_right(name, g):
    call = CALLS[name](g)
    want = call()
    nq.device_error()
    gave_up = 0
    for _ in range(20):
        limited(1, call)
        got = [call() for _ in range(3)]
        try:
            nq.device_error()
        except nq.NqError as e:
            assert e.status == -7
            gave_up += 1
        assert all(same(y, want) for y in got)
    assert gave_up
    nq.device_error()


@pytest.mark.parametrize("name", [n for n in CALLS if not n.startswith("experts")])
def test_a_long_call_ahead_is_not_charged_to_the_next(name, g):
    """A dense call whose blocks start while the call ahead of it still runs, for longer than the limit of a wait."""
    call = CALLS[name](g)
    want = call()
    x, xs = ref.activations(100, 1 << 19, g)
    w, ws = ref.weights(1, 200, 1 << 19, g)
    xs *= 2.0 ** -12
    ends = torch.tensor([0, 100], dtype=torch.int32, device="cuda")
    ahead = lambda: nq.gemm_fp8_experts(x, xs, w, ws, ends)   # one tile of 4096 blocks of K: some 2 ms on one SM  # noqa: E731
    ahead()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    ahead()
    end.record()
    nq.device_error()
    assert begin.elapsed_time(end) > 1.0
    for _ in range(5):
        ahead()
        got = limited(300_000, call)
        nq.device_error()
        assert same(got, want)
