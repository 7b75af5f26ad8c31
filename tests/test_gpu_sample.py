"""Sampling against its definition in 64 bits, row by row. On random rows a token is accepted if an
error of 1e-6 (relative: fp32 scores, masses of fp32 exponentials) could choose it, which leaves
one token for nearly all of them; exact ties, cuts inside ties and edge settings are made on
purpose, with values on which both sides are exact."""
import math

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def nq():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from weight_only_groupwise_gb300 import build
    build.build()
    from weight_only_groupwise_gb300 import nq
    return nq


def pick(row, noise, t, k, p, m, slack=0.0):
    """The tokens that may be chosen: one, or with `slack` every one that a relative error of that
    size in a mass, a threshold or a score could choose instead."""
    row = np.where(np.isnan(row), -np.inf, row)
    ids = np.lexsort((np.arange(row.size), -row))
    ids = ids[row[ids] > -np.inf]
    if not ids.size:
        return {-1}
    if not t > 0:
        return {int(ids[0])}
    if k > 0:
        ids = ids[:k]
    with np.errstate(invalid="ignore", divide="ignore"):
        d = np.where(row[ids] == row[ids[0]], 0.0, (row[ids] - row[ids[0]]) / t)
        w, found = np.exp(d), set()
        before = np.concatenate([[0.0], np.cumsum(w)[:-1]])
        for off in {-slack, 0.0, slack}:
            n = ids.size
            if p < 1:
                n = max(1, int((before < p * w.sum() * (1 + off)).sum()))
            for off_m in {-slack, 0.0, slack}:
                if m > 0:
                    n_m = max(1, min(n, int((d >= math.log(min(m, 1.0)) * (1 + off_m)).sum())))
                else:
                    n_m = n
                score = d[:n_m] - np.log(noise[ids[:n_m]])
                best = score == score.max()
                if slack:
                    best |= score >= score.max() - 2 * slack * (1 + abs(score.max()))
                found |= set(ids[:n_m][best].tolist()) if slack else {int(ids[:n_m][best].min())}
    return found


def settings(B, t, k, p, m):
    f = lambda x: torch.tensor(np.broadcast_to(np.asarray(x, np.float32), B).copy(), device="cuda")  # noqa: E731
    return {"temperature": f(t), "top_p": f(p), "min_p": f(m),
            "top_k": torch.tensor(np.broadcast_to(np.asarray(k, np.int32), B).copy(), device="cuda")}


def check(nq, logits, noise, s, sure=False):
    got = nq.sample(logits, noise, **s).cpu().numpy()
    x, e = logits.double().cpu().numpy(), noise.double().cpu().numpy()
    st = [s[n].double().cpu().numpy() if s.get(n) is not None else np.full(len(x), d)
          for n, d in (("temperature", 1.0), ("top_k", 0), ("top_p", 1.0), ("min_p", 0.0))]
    for i in range(len(x)):
        may = pick(x[i], e[i], st[0][i], int(st[1][i]), st[2][i], st[3][i], 0.0 if sure else 1e-6)
        assert int(got[i]) in may, (i, [float(c[i]) for c in st])
    return got


def rows(B, V, dtype, seed, spread=2.2, hot=20):
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((B, V), device="cuda", generator=g) * spread
    if hot:
        at = torch.randint(0, V, (B, hot), device="cuda", generator=g)
        x.scatter_add_(1, at, torch.rand((B, hot), device="cuda", generator=g) * 12)
    x[:, ::97] = -math.inf
    return x.to(dtype), torch.empty((B, V), device="cuda").exponential_(generator=g)


DTYPES = [torch.bfloat16, torch.float16, torch.float32]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 2, 7, 8, 9, 100, 127, 1000, 4097, 32001, 152064])
def test_mixed_settings(nq, V, dtype):
    B = 24
    x, e = rows(B, V, dtype, V)
    r = np.random.default_rng(V)
    check(nq, x, e, settings(B, r.choice([0.0, 0.3, 0.7, 1.0, 1.5, 4.0], B), r.choice([0, 1, 5, 50, 700, 5000], B),
                             r.choice([1.0, 0.1, 0.9, 0.99], B), r.choice([0.0, 0.0, 0.05, 0.3], B)))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("t,k,p,m", [(1.0, 0, 1.0, 0.0), (0.7, 50, 0.9, 0.0), (1.0, 0, 0.95, 0.0), (1.0, 20000, 1.0, 0.0),
                                     (2.0, 0, 0.999, 0.0), (0.2, 30000, 0.99, 0.0), (1.0, 0, 1.0, 0.1),
                                     (3.0, 9000, 0.7, 0.01), (100.0, 0, 0.5, 0.0), (0.01, 0, 0.9, 0.0)])
def test_cuts_few_and_many(nq, dtype, t, k, p, m):
    x, e = rows(6, 50257, dtype, k + 1, hot=0)
    check(nq, x, e, settings(6, t, k, p, m))


@pytest.mark.parametrize("dtype", DTYPES)
def test_rows_shorter_than_their_blocks(nq, dtype):
    """Every length up to a few chunks, at every alignment: blocks without tokens take no part."""
    for V in range(1, 140, 3):
        wide, e = rows(8, V + 8, dtype, V, hot=0)
        for off in (0, 3):
            x = wide[:, off:off + V]
            check(nq, x, e[:, off:off + V], settings(8, [1.0, 0.3, 2.0, 100.0] * 2, [0, V, 0, V - 1] * 2, [1.0] * 4 + [0.9] * 4, 0.0))


def test_equal_logits_are_cut_by_index(nq):
    """All logits equal: top-k and top-p cut inside one tie, whose weights are exactly 1."""
    V = 20000
    for dtype in DTYPES:
        x = torch.full((8, V), 1.5, device="cuda", dtype=dtype)
        e = torch.empty((8, V), device="cuda").exponential_()
        got = check(nq, x, e, settings(8, 1.0, [0, 1, 2, 17, 1024, 1025, 9999, 20000], 1.0, 0.0), sure=True)
        assert got[1] == 0 and got[3] < 17 and got[6] < 9999
        got = check(nq, x, e, settings(8, 1.0, [0] * 4 + [1000] * 4, [0.25, 0.5, 0.125, 0.0] * 2, 0.0), sure=True)
        assert (got < [5000, 10000, 2500, 1, 250, 500, 125, 1]).all()


def test_few_levels_with_many_ties(nq):
    V = 40000
    g = torch.Generator(device="cuda").manual_seed(3)
    x = torch.randint(0, 4, (12, V), device="cuda", generator=g).float()
    e = torch.empty((12, V), device="cuda").exponential_(generator=g)
    k = [1, 100, 5000, 9000, 10500, 15000, 20000, 25000, 30000, 39999, 40000, 50000]
    for dtype in DTYPES:
        check(nq, x.to(dtype), e, settings(12, 1.0, k, 1.0, 0.0))
        check(nq, x.to(dtype), e, settings(12, 1.0, k, 0.7, 0.0))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [4097, 20000, 60000])
def test_scores_that_grow_with_the_rank(nq, V, dtype):
    """The worst noise for a choice by trial: every set's best token is its last in the row's order."""
    x, _ = rows(10, V, dtype, V + 3)
    order = torch.argsort(x.double(), dim=1, descending=True, stable=True)
    place = torch.empty_like(order).scatter_(1, order, torch.arange(V, device="cuda").expand(10, V).contiguous())
    score = place.double() * (20 / V)
    t = 1.25
    e = torch.exp((x.double() - x.double().amax(1, keepdim=True)).clamp(min=-60) / t - score).float()
    k = [0, 0, 0, 300, 3000, 5000, V - 5, 700, 3000, V - 1]
    p = [0.5, 0.97, 0.999, 1.0, 1.0, 1.0, 1.0, 0.9, 0.5, 0.99]
    got = nq.sample(x, e, **settings(10, t, k, p, 0.0)).cpu().numpy()
    d = ((x.double().gather(1, order) - x.double().amax(1, keepdim=True)) / t).cpu().numpy()
    place = place.cpu().numpy()
    for i in range(10):
        n = int((d[i] > -math.inf).sum())
        n = min(n, k[i]) if k[i] else n
        w = np.exp(d[i, :n])
        before, total = np.cumsum(w) - w, w.sum()
        # the last kept token, whatever an error of 1e-6 makes of the share
        least, most = (int((before < np.float32(p[i]) * total * f).sum()) if p[i] < 1 else n for f in (1 - 1e-6, 1 + 1e-6))
        assert least - 1 <= place[i, got[i]] <= most - 1, (i, least, most, place[i, got[i]])


def test_equal_scores_take_the_lowest_index(nq):
    x = torch.zeros((2, 5000), device="cuda")
    e = torch.ones((2, 5000), device="cuda")
    e[0, [700, 4100, 77]] = 0.25
    assert nq.sample(x, e).tolist() == [77, 0]
    assert nq.sample(x, e, top_k=torch.tensor([50, 3], device="cuda", dtype=torch.int32)).tolist() == [0, 0]


def test_greedy_takes_the_first_maximum(nq):
    x, e = rows(5, 3001, torch.float32, 1)
    x[:, [40, 2000, 2999]] = 50.0
    s = settings(5, [0.0, -1.0, math.nan, 0.0, 1e-30], 0, 1.0, 0.0)
    e[:, 40] = 1e-3                       # the last row: only the three maxima have mass
    assert nq.sample(x, e, **s).tolist() == [40] * 5
    assert nq.sample(x, torch.full_like(e, math.nan), **settings(5, 0.0, 7, 0.5, 0.1)).tolist() == [40] * 5


def test_infinities_and_nan(nq):
    V = 1500
    x = torch.zeros((7, V), device="cuda")
    e = torch.ones_like(x)
    x[0] = -math.inf                                    # nothing to choose
    x[1] = math.nan
    x[2, :] = -math.inf
    x[2, 1234] = -3e38                                  # one candidate
    x[3, 700] = math.inf                                # all the mass on two tokens
    x[3, 20] = math.inf
    e[3, 700] = 0.5
    x[4, ::2] = math.nan                                # NaN is never taken
    e[4, ::2] = 1e-6
    e[4, 333] = 0.01
    x[5, 10:] = -math.inf
    e[5, 10:] = 1e-30
    e[5, 4] = 0.1
    x[6, :] = -0.0                                      # equal to +0: the index decides
    x[6, 900] = 0.0
    s = settings(7, 1.0, 0, 1.0, 0.0)
    want = [-1, -1, 1234, 700, 333, 4, 0]
    assert nq.sample(x, e, **s).tolist() == want
    assert nq.sample(x, e, **settings(7, 1.0, 0, 0.9999999, 0.0)).tolist() == want
    want_k = [-1, -1, 1234, 700, 1, 4, 0]
    assert nq.sample(x, e, **settings(7, 1.0, 5, 1.0, 0.0)).tolist() == want_k
    assert nq.sample(x, e, **settings(7, 0.0, 0, 1.0, 0.0)).tolist() == [-1, -1, 1234, 20, 1, 0, 0]


def test_settings_out_of_range_and_none(nq):
    x, e = rows(4, 2000, torch.float32, 5)
    plain = nq.sample(x, e)
    check(nq, x, e, {})
    assert torch.equal(plain, nq.sample(x, e, **settings(4, 1.0, [-5, 2000, 2 ** 31 - 1, 0], [1.0, 2.0, math.nan, math.inf], [-1.0, 0.0, math.nan, 0.0])))
    first = x.argmax(1).int()
    assert torch.equal(first, nq.sample(x, e, **settings(4, 1.0, 0, [0.0, -1.0, 1e-30, 1.0], [0.0, 0.0, 0.0, 5.0])))


def test_strides_alignment_and_streams(nq):
    x, e = rows(6, 5003, torch.bfloat16, 6)
    s = settings(6, 0.8, 40, 0.9, 0.0)
    want = nq.sample(x, e, **s)
    for off in range(1, 9):
        wide = torch.full((6, 5003 + 21), 99.0, device="cuda", dtype=torch.bfloat16)
        wide[:, off:off + 5003] = x
        noisy = torch.zeros((6, 5003 + 21), device="cuda")
        noisy[:, off:off + 5003] = e
        assert torch.equal(want, nq.sample(wide[:, off:off + 5003], noisy[:, off:off + 5003], **s))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = nq.sample(x, e, **s)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(want, got)


def test_largest_vocabulary_and_limits(nq):
    from weight_only_groupwise_gb300.nq import NqError
    for dtype in (torch.float32, torch.bfloat16):
        x, e = rows(2, 524160, dtype, 8)
        check(nq, x, e, settings(2, 1.0, [0, 60], [0.9, 0.95], 0.0))
    with pytest.raises(NqError) as err:
        nq.sample(torch.zeros((1, 524161), device="cuda"), torch.ones((1, 524161), device="cuda"))
    assert err.value.status == -2
    assert nq.sample(torch.zeros((0, 10), device="cuda"), torch.ones((0, 10), device="cuda")).numel() == 0


def test_frequencies(nq):
    """The kept tokens are drawn in proportion to exp(l / T): 200000 draws, five standard deviations."""
    n, t = 200000, 0.7
    l = torch.tensor([1.0, 0.5, 0.0, -1.0, -6.0, 0.9], device="cuda")
    e = torch.empty((n, 6), device="cuda").exponential_(generator=torch.Generator(device="cuda").manual_seed(9))
    got = nq.sample(l.expand(n, 6).contiguous(), e, **settings(n, t, 4, 1.0, 0.0))
    w = torch.softmax(torch.tensor([1.0, 0.5, 0.0, -math.inf, -math.inf, 0.9], dtype=torch.float64) / t, 0)
    seen = torch.bincount(got.long(), minlength=6).double().cpu() / n
    assert ((seen - w).abs() <= 5 * (w * (1 - w) / n).sqrt()).all()


def test_refusals(nq):
    from weight_only_groupwise_gb300.nq import NqError
    x, e = rows(2, 64, torch.float32, 1)
    with pytest.raises(NqError) as err:
        nq.sample(x, e, out=e.view(torch.int32)[0, :2])
    assert err.value.status == -4
    for bad in ({"logits": x.double()}, {"logits": x.t()}, {"noise": e[:1]}, {"noise": e.half()}, {"top_k": torch.zeros(2, device="cuda")},
                {"temperature": torch.ones(3, device="cuda")}, {"logits": x.cpu()}):
        a = {"logits": x, "noise": e} | bad
        with pytest.raises(ValueError):
            nq.sample(a.pop("logits"), a.pop("noise"), **a)
