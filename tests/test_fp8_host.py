"""Argument checks of the 8-bit products, the router and the combination: all run on the host, before any CUDA call, and return the
documented status. Fake device addresses are fine here. No GPU."""
import pytest

from tests.test_step_host import A, L, gpu, passes  # noqa: F401
from weight_only_groupwise_gb300 import nq as nqmod

NULL, SHAPE, ALIGN, ALIAS = -1, -2, -3, -4
BF16, FP16, FP32, E4M3 = 0, 1, 2, 3
HUGE = 1 << 61


def quant(L, x=A, dtype=BF16, xs=1024, rows=50, K=1000 // 16 * 16, codes=2 * A, cs=1024, scales=3 * A, ss=8):  # noqa: F811
    return L.nq_quant_fp8(x, dtype, xs, rows, K, codes, cs, scales, ss, 0)


def rows_of(codes=A, scales=2 * A, stride=512, ss=4, rows=50):
    return nqmod._F8_ROWS.pack(codes, scales, stride, ss, rows)


def weight(codes=3 * A, scales=4 * A, row=512, expert=512 * 300, srow=4, sexpert=12):
    return nqmod._F8_WEIGHT.pack(codes, scales, row, expert, srow, sexpert)


def out(data=7 * A, scales=8 * A, stride=300, ss=3, dtype=BF16):
    return nqmod._F8_OUT.pack(data, scales, stride, ss, dtype)


def gemm(L, x=None, w=None, y=None, K=512, N=300):  # noqa: F811
    return L.nq_gemm_fp8(x or rows_of(), w or weight(), y or out(), K, N, 0)


def swiglu(L, x=None, wg=None, wu=None, y=None, K=512, N=288):  # noqa: F811
    return L.nq_swiglu_fp8(x or rows_of(), wg or weight(), wu or weight(codes=5 * A, scales=6 * A), y or out(), K, N, 0)


def experts(L, x=None, rows=9 * A, M=70, offsets=10 * A, E=5, w=None, y=None, K=512, N=300, scratch=0):  # noqa: F811
    return L.nq_gemm_fp8_experts(x or rows_of(), rows, M, offsets, E, w or weight(), y or out(), K, N, scratch, 0)


def route(L, logits=A, dtype=BF16, stride=64, bias=0, T=40, E=64, k=4, score=0, normalize=1, scale=1.0, ids=2 * A, w=3 * A, offsets=4 * A,  # noqa: F811
          rows=5 * A, slots=6 * A):
    return L.nq_moe_route(logits, dtype, stride, bias, T, E, k, score, normalize, scale, ids, w, offsets, rows, slots, 0)


def combine(L, y=A, dtype=BF16, ys=256, M=100, slots=2 * A, w=3 * A, T=30, k=4, N=256, base=4 * A, bs=256, o=5 * A, os=256):  # noqa: F811
    return L.nq_moe_combine(y, dtype, ys, M, slots, w, T, k, N, base, bs, o, os, 0)


def test_structs_match_the_header():
    assert nqmod._F8_ROWS.size == 40 and nqmod._F8_WEIGHT.size == 48 and nqmod._F8_OUT.size == 40


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), SHAPE), (dict(dtype=-1), SHAPE), (dict(rows=-1), SHAPE), (dict(rows=(1 << 24) + 1), SHAPE), (dict(K=8), SHAPE),
    (dict(K=1000), SHAPE), (dict(K=0), SHAPE), (dict(K=(1 << 20) + 16), SHAPE), (dict(xs=900), SHAPE), (dict(cs=900), SHAPE), (dict(ss=7), SHAPE),
    (dict(xs=HUGE), SHAPE), (dict(ss=HUGE), SHAPE), (dict(x=0), NULL), (dict(codes=0), NULL), (dict(scales=0), NULL), (dict(x=A + 8), ALIGN),
    (dict(xs=1004), ALIGN), (dict(cs=1032), ALIGN), (dict(scales=3 * A + 2), ALIGN), (dict(codes=2 * A + 8), ALIGN), (dict(codes=A), ALIAS),
    (dict(scales=A + 64), ALIAS), (dict(scales=2 * A + 64), ALIAS)])
def test_quant(L, change, status):  # noqa: F811
    assert quant(L, **change) == status


@pytest.mark.parametrize("call", [gemm, swiglu, experts])
@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), SHAPE), (dict(stride=500), SHAPE), (dict(ss=3), SHAPE), (dict(stride=HUGE), SHAPE), (dict(codes=0), NULL), (dict(scales=0), NULL),
    (dict(codes=A + 4), ALIGN), (dict(stride=520), ALIGN), (dict(scales=2 * A + 1), ALIGN), (dict(codes=7 * A + 16), ALIAS), (dict(scales=7 * A), ALIAS)])
def test_rows(L, call, change, status):  # noqa: F811
    assert call(L, x=rows_of(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(row=496), SHAPE), (dict(srow=3), SHAPE), (dict(row=HUGE), SHAPE), (dict(expert=HUGE), SHAPE), (dict(expert=-16), SHAPE),
    (dict(sexpert=-1), SHAPE), (dict(codes=0), NULL), (dict(scales=0), NULL), (dict(codes=3 * A + 8), ALIGN), (dict(row=520), ALIGN), (dict(expert=8), ALIGN),
    (dict(scales=4 * A + 2), ALIGN), (dict(codes=7 * A), ALIAS), (dict(scales=7 * A + 64), ALIAS)])
def test_weights(L, change, status):  # noqa: F811
    assert experts(L, w=weight(**change)) == status
    if not set(change) & {"expert", "sexpert"}:      # one weight has no experts apart
        assert gemm(L, w=weight(**change)) == status
        assert swiglu(L, wg=weight(**change)) == status and swiglu(L, wu=weight(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=FP32), SHAPE), (dict(dtype=4), SHAPE), (dict(stride=280), SHAPE), (dict(stride=HUGE), SHAPE), (dict(data=0), NULL), (dict(data=7 * A + 1), ALIGN),
    (dict(dtype=E4M3, stride=304, ss=2), SHAPE), (dict(dtype=E4M3, stride=296), ALIGN), (dict(dtype=E4M3, stride=304, scales=0), NULL),
    (dict(dtype=E4M3, stride=304, data=7 * A + 8), ALIGN), (dict(dtype=E4M3, stride=304, scales=7 * A + 64), ALIAS), (dict(dtype=E4M3, stride=304, scales=A), ALIAS)])
def test_results(L, change, status):  # noqa: F811
    assert swiglu(L, y=out(**change)) == status


def test_results_of_codes_are_the_swiglu_calls_alone(L):  # noqa: F811
    assert gemm(L, y=out(dtype=E4M3, stride=304)) == SHAPE and experts(L, y=out(dtype=E4M3, stride=304)) == SHAPE
    assert swiglu(L, y=out(dtype=E4M3, stride=304), N=300) == SHAPE          # not a multiple of 16


@pytest.mark.parametrize("change,status", [
    (dict(K=0), SHAPE), (dict(K=500), SHAPE), (dict(N=0), SHAPE), (dict(N=(1 << 20) + 1), SHAPE), (dict(E=0), SHAPE), (dict(E=513), SHAPE), (dict(M=-1), SHAPE),
    (dict(M=(1 << 24) + 1), SHAPE), (dict(rows=0), SHAPE), (dict(offsets=0), NULL), (dict(rows=9 * A + 2), ALIGN), (dict(offsets=10 * A + 1), ALIGN),
    (dict(rows=7 * A), ALIAS), (dict(offsets=7 * A + 4), ALIAS), (dict(scratch=11 * A + 8), ALIGN), (dict(M=10000, scratch=7 * A + 512), ALIAS),
    (dict(M=10000, scratch=A), ALIAS), (dict(M=10000, scratch=3 * A - 64), ALIAS)])
def test_groups(L, change, status):  # noqa: F811
    assert experts(L, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=3), SHAPE), (dict(T=-1), SHAPE), (dict(T=(1 << 20) + 1), SHAPE), (dict(E=0), SHAPE), (dict(E=513, stride=513), SHAPE), (dict(k=0), SHAPE),
    (dict(k=33), SHAPE), (dict(E=3), SHAPE), (dict(stride=63), SHAPE), (dict(stride=HUGE), SHAPE), (dict(score=2), SHAPE), (dict(bias=7 * A), SHAPE),
    (dict(scale=0.0), SHAPE), (dict(scale=float("inf")), SHAPE), (dict(scale=float("nan")), SHAPE), (dict(logits=0), NULL), (dict(ids=0), NULL), (dict(w=0), NULL),
    (dict(offsets=0), NULL), (dict(rows=0), NULL), (dict(slots=0), NULL), (dict(logits=A + 1), ALIGN), (dict(dtype=FP32, logits=A + 2), ALIGN),
    (dict(slots=6 * A + 2), ALIGN), (dict(score=1, bias=7 * A + 2), ALIGN), (dict(ids=A), ALIAS), (dict(rows=6 * A), ALIAS), (dict(score=1, bias=4 * A), ALIAS),
    (dict(offsets=2 * A + 8), ALIAS)])
def test_route(L, change, status):  # noqa: F811
    assert route(L, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(dtype=FP32), SHAPE), (dict(M=-1), SHAPE), (dict(T=-1), SHAPE), (dict(k=0), SHAPE), (dict(k=33), SHAPE), (dict(N=0), SHAPE), (dict(N=252), SHAPE),
    (dict(ys=248), SHAPE), (dict(bs=0), SHAPE), (dict(os=248), SHAPE), (dict(os=HUGE), SHAPE), (dict(ys=HUGE), SHAPE), (dict(bs=HUGE), SHAPE), (dict(y=0), NULL),
    (dict(slots=0), NULL), (dict(w=0), NULL), (dict(o=0), NULL), (dict(y=A + 8), ALIGN), (dict(os=260), ALIGN), (dict(base=4 * A + 2), ALIGN), (dict(w=3 * A + 2), ALIGN),
    (dict(o=A), ALIAS), (dict(o=2 * A), ALIAS), (dict(o=4 * A + 512), ALIAS), (dict(o=4 * A, os=264), ALIAS)])
def test_combine(L, change, status):  # noqa: F811
    assert combine(L, **change) == status


def test_scratch_is_asked_for_where_groups_are_large(L):  # noqa: F811
    for swiglu in (0, 1):
        need = lambda *a: L.nq_fp8_scratch_bytes(*a, swiglu)  # noqa: E731, B023
        assert need(10000, 5, 528) == 10000 * (528 + 4 * 8) and need(64, 64, 512) == need(0, 5, 512) == need(10000, 0, 512) == need(10000, 5, 0) == 0


def test_empty_calls_are_accepted(L):  # noqa: F811
    assert quant(L, rows=0, x=0) == 0 and combine(L, T=0) == 0
    assert gemm(L, x=rows_of(rows=0, codes=0, scales=0)) == 0 and swiglu(L, x=rows_of(rows=0)) == 0 and experts(L, M=0, rows=0) == 0


def test_good_calls_pass_the_checks(L):  # noqa: F811
    if gpu():
        pytest.skip("fake addresses: only where no GPU could be reached")
    assert all(passes(c(L)) for c in (quant, gemm, swiglu, experts, route, combine))
    assert passes(swiglu(L, y=out(dtype=E4M3, stride=304))) and passes(quant(L, dtype=FP32)) and passes(route(L, T=0, logits=0))
    assert passes(experts(L, rows=0, M=50)) and passes(experts(L, M=10000, scratch=11 * A)) and passes(route(L, score=1, bias=7 * A)) and passes(combine(L, o=4 * A)) and passes(combine(L, base=0, bs=0))
    # one row's stride means nothing, nor one expert's
    assert passes(gemm(L, x=rows_of(rows=1, stride=HUGE, ss=HUGE), y=out(stride=HUGE))) and passes(gemm(L, w=weight(expert=HUGE, sexpert=HUGE)))
    assert passes(quant(L, rows=1, xs=HUGE, cs=HUGE, ss=HUGE)) and passes(route(L, T=1, stride=HUGE)) and passes(combine(L, T=1, bs=HUGE, os=HUGE))


def test_scales_of_results_that_have_none_do_not_count(L):  # noqa: F811
    """Results in 16 bits: whatever the field holds."""
    if gpu():
        pytest.skip("fake addresses: only where no GPU could be reached")
    for scales, ss in ((8 * A + 1, 0), (7 * A, -5), (A, HUGE)):
        y = out(scales=scales, ss=ss)
        assert passes(gemm(L, y=y)) and passes(swiglu(L, y=y)) and passes(experts(L, y=y))
