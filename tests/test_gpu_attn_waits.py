"""Paged attention whose waits run out, with other calls right behind it: what an aborted block has asked for arrives before it
leaves."""
import pytest
import torch

from tests.test_gpu_attn import problem, reference
from weight_only_groupwise_gb300 import nq

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_only_groupwise_gb300 import build
    build.build()
    yield
    nq.device_error()


# few key tiles (all of a block's copies asked for at once) and many, single blocks and pairs
@pytest.mark.parametrize("kv,new,dim,heads", [([100, 200, 17], [1, 2, 8], 64, 8), ([3000, 300, 5000], [1, 4, 8], 128, 8),
                                              ([300, 2000], [8, 1], 256, 24), ([900, 400], [700, 200], 256, 24)])
def test_a_call_right_behind_one_that_gave_up_is_right(kv, new, dim, heads):
    p = problem(kv, new, heads, heads // 4 if dim < 256 else 4, dim, 64, torch.bfloat16, seed=dim)
    call = lambda: nq.attn_paged(p["q"], p["k"], p["v"], p["table"], p["q_start"], p["kv"])  # noqa: E731
    want = call()
    ref, bound = reference(p, dim ** -0.5)
    assert bool(((want.double() - ref).abs() <= bound).all())
    nq.device_error()
    gave_up = 0
    for _ in range(20):
        before = nq.wait_limit(1)
        try:
            call()
        finally:
            nq.wait_limit(before)
        got = [call() for _ in range(3)]
        try:
            nq.device_error()
        except nq.NqError as e:
            assert e.status == -7
            gave_up += 1
        assert all(torch.equal(y, want) for y in got)
    assert gave_up
    nq.device_error()
