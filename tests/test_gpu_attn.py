"""Paged attention against its definition in 64 bits: head layouts, lengths from no key to
several tiles, pages, windows with sinks, strides, and cache rows that hold NaN where no token
looks."""
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


BF, FP = torch.bfloat16, torch.float16
ROUND = {BF: 2.0 ** -8, FP: 2.0 ** -11}     # unit roundoff of the type


def problem(old, new, heads, kv_heads, dim, page, dtype, seed=0, spare=3, width_more=0):
    """Requests with `old` cached and `new` new tokens over a shuffled pool whose unused rows are NaN."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    old, new = np.asarray(old), np.asarray(new)
    total = old + new
    blocks = -(-total // page)
    pool = int(blocks.sum()) + spare
    ids = np.random.default_rng(seed).permutation(pool)
    width = max(1, int(blocks.max()) + width_more)
    table = np.full((len(total), width), -1, np.int32)
    at = 0
    k = torch.full((pool, page, kv_heads, dim), math.nan, device="cuda", dtype=dtype)
    v = k.clone()
    keys = []
    for r, n in enumerate(total.tolist()):
        b = int(blocks[r])
        table[r, :b] = ids[at:at + b]
        rows = torch.randn((2, b * page, kv_heads, dim), device="cuda", generator=g).to(dtype)
        keys.append(rows[:, :n])
        rows[:, n:] = math.nan
        mine = torch.as_tensor(ids[at:at + b].copy(), device="cuda")
        if b:
            k[mine] = rows[0].view(b, page, kv_heads, dim)
            v[mine] = rows[1].view(b, page, kv_heads, dim)
        at += b
    q = (torch.randn((int(new.sum()), heads, dim), device="cuda", generator=g) * 2).to(dtype)
    i32 = lambda x: torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")  # noqa: E731
    return {"q": q, "k": k, "v": v, "table": i32(table), "q_start": i32(np.concatenate([[0], np.cumsum(new)])),
            "kv": i32(total), "keys": keys, "old": old, "new": new}


def reference(p, scale, window=0, sinks=0):
    """(output, error bound) in 64 bits: the bound is the output's rounding, the rounding of each
    probability to the 16-bit type (its absolute least step too), and 2^-12 for the fp32 scores."""
    q, dtype = p["q"].double(), p["q"].dtype
    u = ROUND[dtype]
    out, bound = torch.zeros_like(q), torch.zeros_like(q)
    at = 0
    for r, (k, v) in enumerate(p["keys"]):
        n, total = int(p["new"][r]), k.shape[0]
        g = q.shape[1] // k.shape[1]
        pos = torch.arange(total - n, total, device="cuda")[:, None]
        j = torch.arange(total, device="cuda")[None]
        seen = j <= pos
        if window:
            seen &= (j > pos - window) | (j < sinks)
        for h in range(q.shape[1]):
            kk, vv = k[:, h // g].double(), v[:, h // g].double()
            s = (q[at:at + n, h] @ kk.T * scale).masked_fill(~seen, -math.inf)
            w = torch.softmax(s, -1).nan_to_num(0.0)
            o, a = w @ vv, w @ vv.abs()
            out[at:at + n, h] = o
            bound[at:at + n, h] = u * o.abs() + (u + 2.0 ** -12) * a
            if dtype == FP:
                bound[at:at + n, h] += 2.0 ** -24 * (1 + vv.abs().sum(0))
        at += n
    return out, bound + 1e-6


def check(nq, p, window=0, sinks=0, scale=None, **kw):
    scale = p["q"].shape[2] ** -0.5 if scale is None else scale
    out = nq.attn_paged(p["q"], p["k"], p["v"], p["table"], p["q_start"], p["kv"], scale=scale, window=window,
                        sinks=sinks, **kw)
    nq.device_error()
    ref, bound = reference(p, scale, window, sinks)
    err = (out.double() - ref).abs()
    assert torch.isfinite(out).all(), "not finite"
    worst = (err / bound).max().item() if out.numel() else 0.0
    assert worst <= 1.0, f"error {worst:.3f} of the bound"
    return out


LAYOUTS = [(24, 4, 256), (32, 8, 128), (16, 16, 64), (14, 2, 128), (10, 1, 256), (9, 3, 64), (1, 1, 128)]


@pytest.mark.parametrize("heads,kv_heads,dim", LAYOUTS)
@pytest.mark.parametrize("dtype", [BF, FP])
def test_layouts_and_types(nq, heads, kv_heads, dim, dtype):
    p = problem([0, 5, 300, 127, 1000], [7, 1, 40, 1, 3], heads, kv_heads, dim, 64, dtype, seed=heads + dim)
    check(nq, p)


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_pages(nq, page, dim):
    p = problem([page - 1, page, 3 * page + 1, 517], [1, 1, 2, 9], 4, 2, dim, page, BF, seed=page + dim, width_more=2)
    check(nq, p)


@pytest.mark.parametrize("total", [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 256, 257, 1025])
def test_lengths_of_one_token(nq, total):
    p = problem([total - 1], [1], 6, 1, 256, 64, BF, seed=total)
    check(nq, p)


@pytest.mark.parametrize("new", [1, 2, 21, 22, 43, 64, 127, 128, 129, 500])
def test_prompts_without_a_cache(nq, new):
    p = problem([0], [new], 12, 2, 128, 32, BF, seed=new)
    check(nq, p)


@pytest.mark.parametrize("dim,page", [(256, 64), (128, 16), (64, 32)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (17, 4), (128, 0), (128, 128), (200, 130), (300, 500), (4096, 4)])
def test_windows_and_sinks(nq, dim, page, window, sinks):
    p = problem([900, 0, 130, 1], [70, 33, 1, 1], 6, 2, dim, page, BF, seed=window + sinks)
    check(nq, p, window, sinks)


def test_window_pages_given_back(nq):
    """Entries of pages below the window (and past the sinks) may be gone: -1, or rows of NaN."""
    p = problem([2000], [5], 8, 2, 128, 16, FP, seed=5)
    first = (2000 - 100 + 1) // 16           # the first page of the first token's window
    gone = p["table"][0, 1:first].long()
    p["k"][gone] = math.nan
    p["v"][gone] = math.nan
    check(nq, p, window=100, sinks=3)
    p["table"][0, 1:first] = -1
    check(nq, p, window=100, sinks=3)


@pytest.mark.parametrize("dim,page", [(256, 64), (128, 16), (128, 256), (64, 128)])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (37, 5), (128, 16), (130, 70), (256, 128), (300, 200)])
def test_rows_between_sinks_and_window_hold_nan(nq, dim, page, window, sinks):
    """Rows that no new token sees, in pages with seen ones and of their own; the latter's entries name a NaN page."""
    old, new = [700, 513, 250, 37, 1000, 384], [1, 2, 1, 3, 8, 1]
    p = problem(old, new, 8, 2, dim, page, BF, seed=window + page)
    pad = int(next(i for i in range(p["k"].shape[0]) if not (p["table"] == i).any()))      # a spare page: all NaN
    assert p["v"][pad].isnan().all()
    for r, (have, n) in enumerate(zip(old, new)):
        lo = have - window + 1          # the first new token's first key
        for key in range(sinks, max(sinks, lo)):
            at = (int(p["table"][r, key // page]), key % page)
            p["k"][at] = math.nan
            p["v"][at] = math.nan
        for b in range(-(-(have + n) // page)):
            if b * page >= sinks and (b + 1) * page <= lo:
                p["table"][r, b] = pad
    check(nq, p, window, sinks)


def test_long_split_and_many_tiles(nq):
    """One request over every block of the grid, and prompts of several query tiles."""
    check(nq, problem([40000], [1], 6, 1, 256, 64, BF, seed=1))
    check(nq, problem([9000, 3], [8, 8], 24, 4, 256, 64, BF, seed=2))
    check(nq, problem([1000, 17, 0], [400, 200, 333], 8, 2, 128, 16, BF, seed=3))


@pytest.mark.parametrize("heads,kv_heads,dim,page,dtype", [(32, 8, 128, 16, FP), (16, 16, 64, 32, BF), (12, 2, 256, 64, BF)])
def test_many_requests(nq, heads, kv_heads, dim, page, dtype):
    """More requests than a warp has lanes, each of many key tiles and several to a block."""
    r = np.random.default_rng(dim)
    p = problem(r.integers(0, 6000, 70), r.integers(0, 4, 70), heads, kv_heads, dim, page, dtype, seed=dim)
    first = check(nq, p)
    for _ in range(20):
        assert torch.equal(first, nq.attn_paged(p["q"], p["k"], p["v"], p["table"], p["q_start"], p["kv"]))
    nq.device_error()


@pytest.mark.parametrize("old,new,heads,kv_heads,page,dtype", [
    ([0], [700], 24, 4, 64, BF), ([0], [300], 64, 1, 64, FP), ([700], [800], 24, 4, 16, BF),
    ([100, 0, 5000], [250, 129, 400], 24, 4, 64, BF), ([3000], [2100], 8, 8, 256, BF), ([1], [1100], 16, 2, 32, FP),
    ([64, 900, 0, 30], [1200, 1, 0, 500], 10, 1, 128, BF), ([20000], [700], 24, 4, 64, BF)])
def test_prompts_of_256_columns(nq, old, new, heads, kv_heads, page, dtype):
    """Calls large enough that two blocks share a query tile."""
    p = problem(old, new, heads, kv_heads, 256, page, dtype, seed=sum(new))
    first = check(nq, p)
    assert torch.equal(first, check(nq, p))


@pytest.mark.parametrize("window,sinks", [(1, 0), (100, 4), (300, 130), (4096, 0), (4097, 4), (5000, 200)])
def test_prompts_of_256_columns_with_windows(nq, window, sinks):
    p = problem([6000, 0], [500, 300], 24, 4, 256, 64, BF, seed=window)
    check(nq, p, window, sinks)


def test_large_scores_and_rescaling(nq):
    """Scores that grow along the keys: the running maximum moves in every tile."""
    p = problem([1500], [6], 4, 1, 128, 64, BF, seed=9)
    ramp = torch.linspace(0.1, 6, 1506, device="cuda")[:, None, None]
    k = (p["keys"][0][0].float().abs() * ramp).to(BF)
    ids = p["table"][0].long()
    whole = torch.full((ids.numel() * 64, 1, 128), math.nan, device="cuda", dtype=BF)
    whole[:1506] = k
    p["k"][ids] = whole.view(-1, 64, 1, 128)
    p["keys"][0] = (k, p["keys"][0][1])
    p["q"] = p["q"].abs()
    check(nq, p)


def test_empty_requests_rows_and_padding(nq):
    p = problem([10, 0, 20], [3, 0, 2], 4, 2, 128, 32, BF, seed=4)
    q = torch.cat([p["q"], p["q"]])                       # five rows past the last request
    out = torch.full_like(q, 7.0)
    nq.attn_paged(q, p["k"], p["v"], p["table"], p["q_start"], p["kv"], out=out)
    ref, bound = reference(p, 128 ** -0.5)
    assert ((out[:5].double() - ref).abs() <= bound).all()
    assert (out[5:] == 0).all()
    # a refused request (no keys) and one with fewer keys than new tokens: zeros where nothing is seen
    kv = p["kv"].clone()
    kv[0], kv[2] = 0, 1
    out = nq.attn_paged(p["q"], p["k"], p["v"], p["table"], p["q_start"], kv)
    assert (out[:4] == 0).all()
    assert torch.isfinite(out[4]).all() and (out[4] != 0).any()
    none = nq.attn_paged(p["q"], p["k"], p["v"], p["table"], p["q_start"], torch.zeros_like(kv))
    assert (none == 0).all()


def test_strides_and_cache_orders(nq):
    p = problem([300, 50], [5, 9], 8, 2, 128, 32, BF, seed=6)
    want = check(nq, p)
    wide = torch.full((14, 3, 8, 128), 3.0, device="cuda", dtype=BF)
    wide[:, 1] = p["q"]
    got = torch.zeros((14, 2, 8, 128), device="cuda", dtype=BF)
    table = torch.full((2, p["table"].shape[1] + 5), -1, device="cuda", dtype=torch.int32)
    table[:, :p["table"].shape[1]] = p["table"]
    heads_first = [x.transpose(1, 2).contiguous().transpose(1, 2) for x in (p["k"], p["v"])]
    both = torch.stack([p["k"], p["v"]], 1)
    for k, v in (heads_first, (both[:, 0], both[:, 1])):
        nq.attn_paged(wide[:, 1], k, v, table[:, :p["table"].shape[1]], p["q_start"], p["kv"], out=got[:, 1])
        assert torch.equal(got[:, 1], want) and (got[:, 0] == 0).all()


def test_repeatable_and_on_another_stream(nq):
    p = problem([5000, 100], [8, 8], 24, 4, 256, 64, BF, seed=7)
    want = check(nq, p)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = nq.attn_paged(p["q"], p["k"], p["v"], p["table"], p["q_start"], p["kv"])
    torch.cuda.current_stream().wait_stream(s)
    assert torch.equal(got, want)


def test_calls_in_a_row_share_the_workspace(nq):
    """Calls that split their tiles differently, one after the other without a wait: the same bits as alone."""
    shapes = [([4100], [1], 24, 4, 256, 64), ([9000, 300], [2, 1], 8, 2, 128, 16), ([700] * 5, [60] * 5, 16, 16, 64, 32),
              ([100], [900], 12, 2, 256, 64), ([20000], [1], 32, 8, 128, 16), ([5], [3], 8, 8, 128, 32),
              ([3000] * 40, [1] * 40, 10, 1, 256, 128)]
    todo = []
    for i, (old, new, heads, kv_heads, dim, page) in enumerate(shapes):
        p = problem(old, new, heads, kv_heads, dim, page, BF if i % 2 else FP, seed=i)
        args = (p["q"], p["k"], p["v"], p["table"], p["q_start"], p["kv"])
        alone = nq.attn_paged(*args, scale=dim ** -0.5)
        torch.cuda.synchronize()
        todo.append((args, dim ** -0.5, alone, torch.empty_like(p["q"])))
    order = np.random.default_rng(2).integers(0, len(todo), 200)
    for i in order.tolist():
        args, scale, _, out = todo[i]
        nq.attn_paged(*args, scale=scale, out=out)
    nq.device_error()
    for args, scale, alone, out in todo:
        assert torch.equal(alone, out)


def test_in_a_graph_with_growing_lengths(nq):
    p = problem([200], [1], 8, 2, 128, 32, BF, seed=8)
    nq.attn_reserve()
    out = torch.empty_like(p["q"])
    nq.attn_paged(p["q"], p["k"], p["v"], p["table"], p["q_start"], p["kv"], out=out)
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        nq.attn_paged(p["q"], p["k"], p["v"], p["table"], p["q_start"], p["kv"], out=out)
    for kv in (201, 77, 1):
        p["kv"].fill_(kv)
        g.replay()
        cut = dict(p, keys=[(p["keys"][0][0][:kv], p["keys"][0][1][:kv])])
        ref, bound = reference(cut, 128 ** -0.5)
        assert ((out.double() - ref).abs() <= bound).all()


def test_block_ids_outside_the_cache_read_as_zeros(nq):
    p = problem([100], [1], 2, 1, 64, 32, BF, seed=10)
    p["table"][0, 1] = 10 ** 9
    out = nq.attn_paged(p["q"], p["k"], p["v"], p["table"], p["q_start"], p["kv"])
    k, v = p["keys"][0]
    k[32:64], v[32:64] = 0, 0
    ref, bound = reference(dict(p, keys=[(k, v)]), 64 ** -0.5)
    assert ((out.double() - ref).abs() <= bound).all()


def test_offsets_past_32_bits(nq):
    """A cache of more than 2^32 bytes, its last blocks in use."""
    pool, page, dim = 2 ** 32 // (64 * 256 * 2) + 40, 64, 256
    k = torch.zeros((pool, page, 1, dim), device="cuda", dtype=BF)
    v = torch.zeros_like(k)
    small = problem([150], [2], 4, 1, dim, page, BF, seed=11)
    ids = small["table"][0].long()
    far = torch.arange(pool - ids.numel(), pool, device="cuda")
    k[far], v[far] = small["k"][ids], small["v"][ids]
    small.update(k=k, v=v, table=far[None].to(torch.int32))
    check(nq, small)


def test_refusals(nq):
    from weight_only_groupwise_gb300.nq import NqError
    p = problem([20], [2], 4, 2, 64, 32, BF, seed=12)
    call = lambda **kw: nq.attn_paged(*[kw.pop(n, p[n]) for n in ("q", "k", "v", "table", "q_start", "kv")], **kw)  # noqa: E731
    for bad in ({"scale": 0.0}, {"scale": -1.0}, {"scale": math.inf}, {"scale": math.nan}, {"sinks": 4}, {"window": -1},
                {"q": p["q"][:, :3]}):
        with pytest.raises(NqError) as e:
            call(**bad)
        assert e.value.status == -2, bad
    with pytest.raises(NqError) as e:
        call(out=p["q"])
    assert e.value.status == -4
    with pytest.raises(NqError) as e:            # not 16-byte aligned
        call(q=torch.zeros(2 * 4 * 64 + 1, device="cuda", dtype=BF)[1:].view(2, 4, 64))
    assert e.value.status == -3
    for bad in ({"q": p["q"].to(FP)}, {"q": p["q"].transpose(0, 1)}, {"k": p["k"].float(), "v": p["v"].float()},
                {"v": p["v"].transpose(1, 2).contiguous().transpose(1, 2)}, {"kv": p["kv"].long()},
                {"table": p["table"].long()}, {"q_start": p["q_start"][:1]}, {"q": p["q"].cpu()}):
        with pytest.raises(ValueError):
            call(**bad)
