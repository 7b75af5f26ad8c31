"""Strides of the serving-step calls whose spans no memory holds: refused before they overflow an alias check or an
address. All on the host, with fake addresses. No GPU."""
import pytest

from tests.test_step_host import A, L, SHAPE, append, attn, cache, gpu, passes, sample, tables  # noqa: F401

HUGE = 1 << 61       # times a handful of rows and two bytes: past 64 bits
BIG = 1 << 40


@pytest.mark.parametrize("stride", [HUGE, BIG])
def test_rows_too_far_apart(L, stride):  # noqa: F811
    assert sample(L, stride=stride, B=5) == SHAPE and sample(L, ns=stride, B=5) == SHAPE
    assert append(L, ks=stride) == SHAPE and append(L, vs=stride) == SHAPE
    assert attn(L, qs=stride) == SHAPE and attn(L, os=stride) == SHAPE and attn(L, ts=stride) == SHAPE
    assert tables(L, ts=stride) == SHAPE


def test_caches_of_too_many_blocks(L):  # noqa: F811
    c = cache(bs=(1 << 38) - 8, blocks=1 << 28)
    assert append(L, c) == SHAPE and attn(L, c) == SHAPE
    assert append(L, cache(bs=1 << 30, blocks=1 << 9)) == SHAPE
    assert append(L, cache(hs=(1 << 38) - 8)) == SHAPE and append(L, cache(rs=(1 << 38) - 8)) == SHAPE
    assert append(L, cache(hs=(1 << 38) - 8, blocks=1)) == SHAPE


def test_one_rows_stride_means_nothing(L):  # noqa: F811
    if gpu():
        pytest.skip("fake addresses: only where no GPU could be reached")
    assert passes(sample(L, stride=HUGE, ns=HUGE, B=1))
    assert passes(append(L, ks=HUGE, vs=HUGE, tokens=1))
    assert passes(attn(L, qs=HUGE, os=HUGE, tokens=1)) and passes(attn(L, ts=HUGE, R=1))
    assert passes(tables(L, ts=HUGE, R=1))
    assert passes(append(L, cache(bs=(1 << 38) - 8, blocks=1)))


def test_the_largest_spans_pass(L):  # noqa: F811
    if gpu():
        pytest.skip("fake addresses: only where no GPU could be reached")
    assert passes(append(L, cache(bs=1 << 29, blocks=1 << 9)))
    assert passes(sample(L, stride=(1 << 38) // 3 - 1000))
