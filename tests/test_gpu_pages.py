"""Page tables and KV append against their definition in plain Python: exact."""
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


def i32(x):
    return torch.as_tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def expected(lens, new, free, num_free, table, page, cap):
    """The definition, one request after another."""
    table = table.copy()
    q_start, kv, pos, slots = [0], [], [], []
    asked = taken = refused = tokens = 0
    for r, (old, n) in enumerate(zip(lens, new)):
        m = max(n, 0)
        first, last = min(tokens, cap), min(tokens + m, cap)
        tokens += m
        q_start.append(last)
        ok = old >= 0 and n >= 0 and old + n <= table.shape[1] * page and tokens <= cap
        have, want = (-(-old // page), -(-(old + m) // page)) if ok else (0, 0)
        asked += want - have
        if not ok or (want > have and asked > num_free):
            refused += 1
            kv.append(0)
            pos += [-1] * (last - first)
            slots += [-1] * (last - first)
            continue
        table[r, have:want] = free[asked - (want - have):asked]
        if want > have:
            taken = asked
        kv.append(old + n)
        for p in range(old, old + n):
            pos.append(p)
            slots.append(int(table[r, p // page]) * page + p % page)
    pos += [-1] * (cap - len(pos))
    slots += [-1] * (cap - len(slots))
    return table, q_start, kv, pos, slots, [q_start[-1], taken, refused]


def run(nq, lens, new, page, max_blocks, free, cap=None, num_free=None, seed=0):
    lens, new = list(map(int, lens)), list(map(int, new))
    cap = sum(max(n, 0) for n in new) if cap is None else cap
    own = [min(max(0, -(-o // page)), max_blocks) for o in lens]
    ids = np.random.default_rng(seed).permutation(sum(own) + free + 100)
    table = np.full((len(lens), max_blocks), -7, np.int32)
    at = free
    for r, b in enumerate(own):
        table[r, :b] = ids[at:at + b]
        at += b
    num_free = free if num_free is None else num_free
    dev = i32(table)
    got = nq.page_tables(i32(lens), i32(new), i32(ids[:free]), i32([num_free]), dev, page, cap)
    want = expected(lens, new, ids[:free], min(num_free, free), table, page, cap)
    for name, g, w in zip(("table", "q_start", "kv_lens", "positions", "slots", "counts"), (dev, *got), want):
        assert np.array_equal(g.cpu().numpy(), np.asarray(w).astype(g.cpu().numpy().dtype)), name
    return got


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("R", [1, 2, 31, 33, 500, 1025, 8192])
def test_random_lengths(nq, page, R):
    g = np.random.default_rng(R + page)
    lens, new = g.integers(0, 700, R), g.integers(0, 40, R)
    run(nq, lens, new, page, 800 // page + 1, int(R * (40 // page + 1)) + 1)


def test_lengths_at_page_edges(nq):
    run(nq, [0, 0, 63, 64, 65, 64, 128, 0, 63], [0, 1, 1, 0, 63, 64, 129, 64, 2], 64, 5, 12)


def test_free_list_runs_short(nq):
    # the third needs more than is left; the fourth needs none and is admitted; the fifth is refused with it
    got = run(nq, [0, 60, 10, 30, 0], [64, 10, 300, 2, 1], 64, 8, 4)
    assert got[4].tolist() == [377, 2, 2]
    run(nq, [0, 0, 0], [64, 64, 64], 64, 8, 0)
    run(nq, [5, 0], [1, 64], 64, 8, 3, num_free=0)
    run(nq, [0, 0], [64, 64], 64, 8, 1, num_free=50)         # never past the list itself


def test_unusable_lengths(nq):
    run(nq, [-1, 3, 100, 2 ** 31 - 5, 7], [4, -2, 60, 10, 5], 16, 10, 40)


def test_tokens_past_the_buffers(nq):
    run(nq, [0, 0, 5, 9], [10, 20, 30, 2], 16, 8, 20, cap=45)
    run(nq, [0, 0], [10, 20], 16, 8, 20, cap=100)
    run(nq, [3], [0], 16, 8, 20, cap=0)
    run(nq, [0, 4], [5, 0], 16, 8, 20, cap=3)


def test_long_prompts(nq):
    run(nq, [0, 1000, 131071], [200000, 1, 70000], 64, 4000, 5000)


def test_no_requests_and_refusals(nq):
    from weight_only_groupwise_gb300.nq import NqError
    none = i32([])
    nq.page_tables(none, none, none, i32([0]), i32(np.zeros((0, 4))), 64, 0)
    for page in (8, 48, 512, 0, -64):
        with pytest.raises(NqError) as e:
            nq.page_tables(i32([0]), i32([4]), i32([1]), i32([1]), i32([[0, 0]]), page, 4)
        assert e.value.status == -2
    lens = i32([0, 0])
    with pytest.raises(NqError) as e:
        nq.page_tables(lens, i32([1, 1]), i32([1, 2]), i32([2]), i32([[0], [0]]), 64, 2,
                       out=(i32([0, 0, 0]), lens, i32([0, 0]), torch.zeros(2, dtype=torch.int64, device="cuda"), i32([0] * 3)))
    assert e.value.status == -4
    with pytest.raises(ValueError):
        nq.page_tables(lens, i32([1]), i32([1, 2]), i32([2]), i32([[0], [0]]), 64, 2)
    with pytest.raises(ValueError):
        nq.page_tables(lens.long(), i32([1, 1]), i32([1, 2]), i32([2]), i32([[0], [0]]), 64, 2)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("tokens,heads,dim,page", [(1, 1, 64, 16), (3, 4, 256, 64), (64, 8, 128, 32), (1000, 3, 64, 128), (517, 2, 256, 256)])
def test_append(nq, tokens, heads, dim, page, dtype):
    g = torch.Generator(device="cuda").manual_seed(tokens)
    blocks = tokens // page + 3
    caches = [torch.randn((blocks, page, heads, dim), device="cuda", generator=g).to(dtype) for _ in range(2)]
    k, v = (torch.randn((tokens, heads, dim), device="cuda", generator=g).to(dtype) for _ in range(2))
    slots = torch.randperm(blocks * page, device="cuda", generator=g)[:tokens]
    slots[::7] = -1
    if tokens > 3:
        slots[1], slots[3] = blocks * page, 2 ** 40          # outside the cache: stored nowhere
    want = [c.clone() for c in caches]
    live = (slots >= 0) & (slots < blocks * page)
    for w, x in zip(want, (k, v)):
        w.view(-1, heads, dim)[slots[live]] = x[live]
    nq.kv_append(k, v, slots, *caches)
    for w, c in zip(want, caches):
        assert torch.equal(w.view(torch.int16), c.view(torch.int16))
    # heads-first caches, one tensor for both, strided tokens
    both = torch.zeros((blocks, 2, heads, page, dim), device="cuda", dtype=dtype)
    wide = torch.stack([k, v], 1)
    nq.kv_append(wide[:, 0], wide[:, 1], slots, both[:, 0].transpose(1, 2), both[:, 1].transpose(1, 2))
    for i, x in enumerate((k, v)):
        flat = both[:, i].transpose(1, 2).reshape(-1, heads, dim)
        assert torch.equal(flat[slots[live]].view(torch.int16), x[live].view(torch.int16))
        assert int((flat != 0).any(-1).any(-1).sum()) == int(live.sum())


def test_append_refusals(nq):
    from weight_only_groupwise_gb300.nq import NqError
    c = torch.zeros((4, 32, 2, 64), device="cuda", dtype=torch.bfloat16)
    d = torch.zeros_like(c)
    k = torch.zeros((3, 2, 64), device="cuda", dtype=torch.bfloat16)
    s = torch.zeros(3, device="cuda", dtype=torch.int64)
    nq.kv_append(k[:0], k[:0], s[:0], c, d)
    with pytest.raises(NqError) as e:
        nq.kv_append(c.view(-1, 2, 64)[:3], k, s, c, d)
    assert e.value.status == -4
    odd = torch.zeros(3 * 128 + 1, device="cuda", dtype=torch.bfloat16)[1:].view(3, 2, 64)
    with pytest.raises(NqError) as e:
        nq.kv_append(odd, k, s, c, d)
    assert e.value.status == -3
    with pytest.raises(NqError) as e:
        nq.kv_append(k, k, s, c[:, :24], d[:, :24])
    assert e.value.status == -2
    for bad in ((k.float(), k, s), (k, k[:2], s), (k, k, s.int()), (k[:, :1], k, s)):
        with pytest.raises(ValueError):
            nq.kv_append(*bad, c, d)
