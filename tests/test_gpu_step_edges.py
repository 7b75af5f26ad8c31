"""Edges of the serving-step calls that were once wrong, each against its definition."""
import math

import numpy as np
import pytest
import torch

from tests.test_gpu_sample import check as check_tokens
from tests.test_gpu_sample import settings

pytestmark = pytest.mark.gpu

BF, FP, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module")
def nq():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from weight_only_groupwise_gb300 import build
    build.build()
    from weight_only_groupwise_gb300 import nq
    return nq


def test_short_rows_over_whole_clusters(nq):
    """Rows so short that a block's first store into another comes at once, over as many clusters as fit, call after
    call: the barrier at the start lets every way through a row end, and the tokens stay the same."""
    g = torch.Generator(device="cuda").manual_seed(1)
    V, B = 65, 38
    x = torch.randn((B, V), device="cuda", generator=g)
    e = torch.empty((B, V), device="cuda").exponential_(generator=g)
    s = settings(B, [1.0, 0.0, 0.7, 1.3] * 9 + [1.0] * 2, [0, 0, 5, 0, 60] * 7 + [0] * 3, [1.0, 0.9, 0.5] * 12 + [0.3] * 2, [0.0, 0.1] * 19)
    want = torch.as_tensor(check_tokens(nq, x, e, s))
    got = [nq.sample(x, e, **s) for _ in range(300)]
    assert all(torch.equal(t.cpu(), want) for t in got)


@pytest.mark.parametrize("dtype,V", [(F32, 400001), (F32, 1001), (BF, 1001), (FP, 30003)])
def test_what_lies_before_a_row_is_no_token(nq, dtype, V):
    """Rows that begin inside a 16-byte chunk, and noise aligned otherwise: the elements before them would win."""
    g = torch.Generator(device="cuda").manual_seed(V)
    for off in (0, 1, 3, 7):
        for noise_off in (8, 9):
            x = torch.full((5, 16 + V + 3), 60.0, device="cuda", dtype=dtype)
            x[:, off + 8:off + 8 + V] = torch.randn((5, V), device="cuda", generator=g).to(dtype)
            e = torch.full((5, 16 + V + 3), 1e-6, device="cuda")
            e[:, noise_off:noise_off + V].exponential_(generator=g)
            check_tokens(nq, x[:, off + 8:off + 8 + V], e[:, noise_off:noise_off + V], settings(5, 1.0, 0, 1.0, 0.0))


@pytest.mark.parametrize("off", [0, 1, 2, 3])
def test_equal_logits_beside_the_ends_of_slices(nq, off):
    """Rows too long for shared memory whose slices end inside a 16-byte chunk: the tokens equal to the race's winner
    are counted once, so that a winner just inside the cut is taken and one just outside is not."""
    V, C = 400001, 8
    step = ((V + C - 1) // C + 15) // 16 * 16
    at = [b + d for b in range(step, V, step) for d in (-1, 0, 1, 2, 3, 4)] + [V - 1, V - 2, 2]
    B = len(at)
    wide = torch.zeros((B, V + 3 + off), device="cuda")       # odd strides: the rows are aligned in every way
    wide = wide[:, :V + 3 + off - (V + 3 + off) % 4] if off == 0 else wide
    x = wide[:, off:off + V]
    e = torch.ones((B, V), device="cuda")
    e[torch.arange(B), at] = 1e-6
    n = torch.tensor(at, device="cuda", dtype=torch.int32)
    assert nq.sample(x, e, top_k=n + 1).tolist() == at
    assert nq.sample(x, e, top_k=n).tolist() == [0] * B
    assert nq.sample(x, e, top_p=((n.double() + 0.5) / V).float()).tolist() == at
    assert nq.sample(x, e, top_p=((n.double() - 0.5) / V).float()).tolist() == [0] * B


@pytest.mark.parametrize("V", [400001, 333335, 524157])
def test_few_levels_in_rows_too_long_for_shared_memory(nq, V):
    g = torch.Generator(device="cuda").manual_seed(V)
    for off in (0, 1, 3):
        x = torch.randint(0, 4, (6, V + 4), device="cuda", generator=g).float()[:, off:off + V]
        e = torch.empty((6, V), device="cuda").exponential_(generator=g)
        check_tokens(nq, x, e, settings(6, 1.0, [5000, V // 2, V - 3, 0, 0, V // 3], [1.0, 1.0, 1.0, 0.9, 0.3, 0.7], 0.0))


def last_kept_wins(x, t=1.0):
    """Noise for which the best token of any set of first tokens is its last: (noise, order, distances)."""
    V = x.shape[1]
    order = torch.argsort(x.double(), dim=1, descending=True, stable=True)
    place = torch.empty_like(order).scatter_(1, order, torch.arange(V, device="cuda").expand(x.shape[0], V).contiguous())
    d = (x.double() - x.double().amax(1, keepdim=True)) / t
    return torch.exp(d - place.double() * (20 / V)).float(), place, d.gather(1, order)


@pytest.mark.parametrize("dtype,V", [(F32, 152064), (F32, 524160), (BF, 152064), (FP, 300007), (F32, 9000)])
def test_shares_cut_beside_and_inside_a_far_tail(nq, dtype, V):
    """A first token, thirty of 1e-5 and a tail that holds 1e-4 in all: shares cut among the thirty (few tokens settle
    them) and inside the tail (trials). The cut may be off by the rounding of the weights alone: V 2^-45 of the first
    token's weight, and what three roundings of exponents up to 31 and the exponential's 2 ulp do to the
    masses behind it, 4e-6 of them."""
    g = torch.Generator(device="cuda").manual_seed(V)
    x = math.log(1e-4 / V) + 0.3 * torch.randn((1, V), device="cuda", generator=g)
    at = torch.randperm(V, device="cuda", generator=g)[:31]
    x[0, at[0]] = 0.0
    x[0, at[1:]] = math.log(1e-5) + 0.2 * torch.rand(30, device="cuda", generator=g)
    x = x.to(dtype)
    e, place, d = last_kept_wins(x)
    w = torch.exp(d[0]).cpu().numpy()
    before, total = np.cumsum(w) - w, w.sum()
    cuts = [0.5 * (before[j] + before[j + 1]) for j in (1, 3, 8, 17, 28)] + [before[31] + f * (total - before[31]) for f in (0.05, 0.3, 0.5, 0.9)]
    p = np.asarray(cuts / total, np.float32)
    B = len(p)
    got = nq.sample(x.expand(B, V).contiguous(), e.expand(B, V).contiguous(), **settings(B, 1.0, 0, p, 0.0))
    for share, token in zip(p.astype(np.float64) * total, got.tolist()):
        off = V * 2.0 ** -45 + 4e-6 * (total - 1)
        least, most = ((before < share + s).sum() - 1 for s in (-off, off))
        assert least <= int(place[0, token]) <= most, (share, least, most, int(place[0, token]))


@pytest.mark.parametrize("dtype,hot", [(F32, 12), (F32, 0), (BF, 0), (BF, 12)])
def test_a_cut_does_not_depend_on_the_batch(nq, dtype, hot):
    """One row with many neighbouring shares, alone (eight blocks a row) and with 255 others (fewer), the
    last kept token winning: the same tokens, as few tokens settle the row or trials do."""
    V, B = 152064, 256
    g = torch.Generator(device="cuda").manual_seed(hot)
    x = torch.randn((1, V), device="cuda", generator=g) * 2.2
    if hot:
        x[0, torch.randperm(V, device="cuda", generator=g)[:hot]] += 14
    x = x.to(dtype)
    e, _, d = last_kept_wins(x)
    p = [0.9]
    for _ in range(B - 1):
        p.append(float(np.nextafter(np.float32(p[-1]), np.float32(1))))
    s = settings(B, 1.0, 0, p, 0.0)
    together = nq.sample(x.expand(B, V).contiguous(), e.expand(B, V).contiguous(), **s)
    alone = torch.cat([nq.sample(x, e, **{n: v[i:i + 1] for n, v in s.items()}) for i in range(B)])
    assert torch.equal(together, alone)


@pytest.mark.parametrize("bad", [0.0, math.nan, math.inf, -1.0, 1e-38])
@pytest.mark.parametrize("dtype,V", [(F32, 152064), (BF, 40007), (F32, 400001), (FP, 300)])
def test_noise_of_tokens_that_are_not_kept_changes_nothing(nq, dtype, V, bad):
    """On each way through a row: few tokens, trials by count and by mass, both cuts, min-p, none."""
    g = torch.Generator(device="cuda").manual_seed(V)
    k = [20, 0, V // 5, 0, V // 3, V // 3, 0, 0]
    p = [0.9, 0.3, 1.0, 0.9, 0.7, 0.8, 1.0, 1.0]
    m = [0.0, 0.0, 0.0, 0.0, 0.0, 0.01, 0.02, 0.0]
    B = len(k)
    x = (torch.randn((B, V), device="cuda", generator=g) * 2.2).to(dtype)
    x[:, ::11] = -math.inf
    x[1, 5:25] = 30.0                       # a share that few tokens hold
    e = torch.empty((B, V), device="cuda").exponential_(generator=g)
    s = settings(B, 1.0, k, p, m)
    want = check_tokens(nq, x, e, s)
    v = x.double()
    order = torch.argsort(v, dim=1, descending=True, stable=True)
    rank = torch.empty_like(order).scatter_(1, order, torch.arange(V, device="cuda").expand(B, V).contiguous())
    d = v - v.amax(1, keepdim=True)
    w = torch.exp(d).gather(1, order)
    n = torch.arange(V, device="cuda")
    for i in range(B):
        kept = (n < k[i]) if k[i] else n >= 0
        mass = (w[i] * kept).cumsum(0)
        # a little more than is kept, so that no cut hangs on a rounding
        kept &= (mass - w[i] < (p[i] + 1e-6) * mass[-1]) | (p[i] >= 1)
        hidden = ~kept[rank[i]] | (v[i] == -math.inf) | (d[i] < (math.log(m[i]) - 1e-5 if m[i] else -math.inf))
        assert hidden.any()
        e[i, hidden] = bad
    assert nq.sample(x, e, **s).tolist() == want.tolist()


def hide(p, page, window, sinks, give_back):
    """NaN in every row that no new token sees; `give_back`: entries of pages without seen rows become -1."""
    for r, (old, n) in enumerate(zip(p["old"].tolist(), p["new"].tolist())):
        if n == 0:
            continue
        lo = old - window + 1
        keys = torch.arange(sinks, max(sinks, lo), device="cuda")
        block = p["table"][r, keys // page].long()
        p["k"][block, keys % page] = math.nan
        p["v"][block, keys % page] = math.nan
        if give_back:
            for b in range(-(-sinks // page), max(0, lo) // page):
                p["table"][r, b] = -1


@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("window,sinks", [(4096, 0), (4097, 4), (4100, 130), (5000, 200), (4224, 300)])
def test_pairs_see_nothing_below_the_window(nq, window, sinks, page):
    """Prompts of 256 columns that two blocks share: rows between the sinks and the window in pages partly seen."""
    from tests.test_gpu_attn import check, problem
    p = problem([6000, 4500, 4090, 0], [500, 300, 77, 130], 24, 4, 256, page, BF, seed=window + page)
    hide(p, page, window, sinks, False)
    first = check(nq, p, window, sinks)
    hide(p, page, window, sinks, True)
    assert torch.equal(first, check(nq, p, window, sinks))


@pytest.mark.parametrize("window,sinks", [(0, 0), (4096, 33)])
def test_pairs_with_more_requests_than_lanes(nq, window, sinks):
    from tests.test_gpu_attn import check, problem
    g = np.random.default_rng(7)
    p = problem(g.choice([0, 5, 63, 700, 4200], 40), g.integers(60, 130, 40), 24, 4, 256, 32, FP, seed=8)
    if window:
        hide(p, 32, window, sinks, True)
    first = check(nq, p, window, sinks)
    for _ in range(10):
        assert torch.equal(first, nq.attn_paged(p["q"], p["k"], p["v"], p["table"], p["q_start"], p["kv"], window=window, sinks=sinks))
    nq.device_error()


def test_page_tables_refuse_lengths_past_31_bits(nq):
    """A table wide enough for 2^31 tokens and more: a request that would pass 2^31 - 1 is refused, one below is not."""
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    most, page = 2 ** 31 - 1, 256
    table = torch.full((4, 2 ** 23 + 1), -7, dtype=torch.int32, device="cuda")
    table[1, 0], table[2, 2 ** 23 - 1], table[3, 2 ** 23 - 1] = 5, 11, 13
    lens, new = i32(most - 4, 3, most - 20, most - 1), i32(10, 2, 10, 1)
    before = table.clone()
    q_start, kv, pos, slots, counts = nq.page_tables(lens, new, i32(1, 2), i32(2), table, page, 23)
    assert q_start.tolist() == [0, 10, 12, 22, 23] and counts.tolist() == [23, 0, 1]
    assert kv.tolist() == [0, 5, most - 10, most]
    assert pos.tolist() == [-1] * 10 + [3, 4] + list(range(most - 20, most - 10)) + [most - 1]
    assert slots.tolist() == [-1] * 10 + [5 * 256 + 3, 5 * 256 + 4] + [11 * 256 + (p % 256) for p in range(most - 20, most - 10)] + [13 * 256 + 254]
    assert torch.equal(table, before)


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [64, 256])
@pytest.mark.parametrize("log2", [20.0, 24.9, 25.1, 27.0])
def test_many_keys_of_small_probability_count(nq, dtype, dim, log2):
    """One key far above 2^18 others (one table row for as many requests as there are SMs, so that a block goes
    through a whole one): V is 0 at it and 1 at the others, so O says what they weigh together. Off by the rounding of
    the others' probability, the same for all (2^-7 where fp16 has six bits left), 2^14 fp32 sums (2^-9) and the output's."""
    keys, page, R = 2 ** 18, 256, 152
    k = torch.zeros((keys // page, page, 1, dim), device="cuda", dtype=dtype)
    v = torch.ones_like(k)
    q = torch.zeros((R, 1, dim), device="cuda", dtype=dtype)
    q[..., 0] = 1.0
    k[0, 5, 0, 0] = 1.0
    v[0, 5] = 0.0
    i32 = lambda x: torch.as_tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.arange(keys // page, device="cuda", dtype=torch.int32).expand(R, -1).contiguous()
    out = nq.attn_paged(q, k, v, table, i32(range(R + 1)), i32([keys] * R), scale=log2 * math.log(2.0)).double()
    nq.device_error()
    rest = (keys - 1) * 2.0 ** -log2
    want = rest / (1.0 + rest)
    assert (out - want).abs().max().item() <= want * (2.0 ** -7 + 2.0 ** -9 + (2.0 ** -8 if dtype is BF else 2.0 ** -11))


@pytest.mark.parametrize("dtype", [F32, BF, FP])
def test_infinite_logits_are_cut_among_themselves(nq, dtype):
    """Three infinite logits among ties: top-k and top-p over trials keep the first, the first two, all."""
    V = 8884
    x = torch.full((6, V), 3.0, device="cuda", dtype=dtype)
    e = torch.full((6, V), 1e-9, device="cuda")
    for i, z in ((4087, 4.0), (4910, 0.8), (8002, 0.4)):
        x[:, i], e[:, i] = math.inf, z
    s = settings(6, 1.3, [60, 60, 60, 3000, 3000, 3000], [-1.0, 0.5, 1.0, 0.3, 0.6, 0.9], 0.0)
    assert nq.sample(x, e, **s).tolist() == [4087, 4910, 8002, 4087, 4910, 8002]


@pytest.mark.parametrize("dim,heads,tile", [(128, 8, 64), (256, 24, 42)])
def test_nan_in_a_seen_row_of_v_stays_in_its_tile(nq, dim, heads, tile):
    """The last token's V row is NaN: it reaches itself and at most its tile's other tokens, 128 / G of one
    block, 256 / G of a pair (rounded down to a block's whole tokens)."""
    from tests.test_gpu_attn import problem, reference
    p = problem([0], [700], heads, 4, dim, 64, BF, seed=dim)
    ref, bound = reference(p, dim ** -0.5)
    p["v"][int(p["table"][0, 699 // 64]), 699 % 64] = math.nan
    out = nq.attn_paged(p["q"], p["k"], p["v"], p["table"], p["q_start"], p["kv"])
    assert out[699].isnan().all()
    first = 700 - tile
    assert ((out[:first].double() - ref[:first]).abs() <= bound[:first]).all()
