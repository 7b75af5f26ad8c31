"""What is measured of the serving-step operators: page tables, KV append, paged attention, sampling.

One decode, verify or prompt step of a paged-cache server takes them in this order, with the projections in
between. `run` makes the framework's calls where `own` is true, else the same results from elementary torch
operations in 32 bits. Sizes are this repository's 27B-class layer (24 query and 4 KV heads of 256, 64-token
pages) or generic.
"""
import math
import random

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def listed():
    return [
        # one decode step of 64 requests: every request adds one token, now and then a page
        {"name": "tables_decode", "op": "tables", "requests": 64, "new": 1, "ctx": 32768, "page": 64, "even": False,
         "free": 1.5, "lens_seed": 1},
        # admission of a queue of prompts into small pages; the pool runs short for the last ones
        {"name": "tables_prompts", "op": "tables", "requests": 509, "new": 500, "ctx": 2048, "page": 16,
         "even": False, "free": 0.9, "lens_seed": 2},
        # a verify round of 8 requests x 8 draft tokens
        {"name": "append_verify", "op": "append", "tokens": 64, "kv_heads": 4, "dim": 256, "page": 64,
         "type": "bf16", "padding": 0},
        # prompt chunks of a busy step, padded as for a captured graph
        {"name": "append_prompt", "op": "append", "tokens": 16381, "kv_heads": 8, "dim": 128, "page": 16,
         "type": "fp16", "padding": 300},
        # a single user's decode step: latency
        {"name": "attn_decode_one", "op": "attn", "requests": 1, "new": 1, "ctx": 4099, "even": True, "heads": 24,
         "kv_heads": 4, "dim": 256, "page": 64, "window": 0, "sinks": 0, "type": "bf16", "lens_seed": 3},
        # verify rounds of several users with long, ragged contexts
        {"name": "attn_verify", "op": "attn", "requests": 8, "new": 8, "ctx": 32768, "even": True, "heads": 24,
         "kv_heads": 4, "dim": 256, "page": 64, "window": 0, "sinks": 0, "type": "bf16", "lens_seed": 4},
        # a batch's decode step over small pages, another head layout and type
        {"name": "attn_decode_batch", "op": "attn", "requests": 64, "new": 1, "ctx": 8192, "even": True, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 16, "window": 0, "sinks": 0, "type": "fp16", "lens_seed": 5},
        # a prompt's next chunk over what is already cached: the compute-bound end
        {"name": "attn_prompt", "op": "attn", "requests": 1, "new": 2048, "ctx": 16384, "even": True, "heads": 24,
         "kv_heads": 4, "dim": 256, "page": 64, "window": 0, "sinks": 0, "type": "bf16", "lens_seed": 6},
        # prompt chunks of a sliding-window layer whose first tokens stay visible
        {"name": "attn_window", "op": "attn", "requests": 3, "new": 700, "ctx": 12000, "even": False, "heads": 32,
         "kv_heads": 8, "dim": 128, "page": 32, "window": 1024, "sinks": 4, "type": "bf16", "lens_seed": 7},
        # one user's next token
        {"name": "sample_one", "op": "sample", "rows": 1, "vocab": 152064, "type": "bf16", "mix": "usual"},
        # every row of a verify round, each request with its own settings
        {"name": "sample_verify", "op": "sample", "rows": 64, "vocab": 152064, "type": "bf16", "mix": "all"},
        # a large batch with 32-bit logits and an odd vocabulary
        {"name": "sample_batch", "op": "sample", "rows": 256, "vocab": 128257, "type": "fp32", "mix": "all"},
    ]


def _log_int(rng, lo, hi):
    n = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    return n + 1 if n == 3072 else n


def draw(rng):
    op = rng.choice(["tables", "append", "attn", "attn", "attn", "sample", "sample"])
    if op == "tables":
        requests = _log_int(rng, 1, 800)
        return {"op": op, "requests": requests, "new": _log_int(rng, 1, max(2, 250000 // requests)),
                "ctx": _log_int(rng, 1, 32768), "page": rng.choice([16, 32, 64, 128, 256]), "even": rng.random() < 0.3,
                "free": rng.choice([0.7, 1.0, 1.5]), "lens_seed": rng.randrange(1 << 30)}
    if op == "append":
        kv_heads, dim = rng.choice([(4, 256), (8, 128), (16, 64), (1, 128), (2, 256), (3, 64)])
        return {"op": op, "tokens": _log_int(rng, 1, 16000), "kv_heads": kv_heads, "dim": dim,
                "page": rng.choice([16, 32, 64, 128]), "type": rng.choice(["bf16", "fp16"]),
                "padding": rng.choice([0, 0, 17])}
    if op == "sample":
        vocab = _log_int(rng, 1000, 200000)
        return {"op": op, "rows": _log_int(rng, 1, min(256, 256 * 128257 // vocab)), "vocab": vocab,
                "type": rng.choice(["bf16", "fp16", "fp32"]), "mix": rng.choice(["usual", "all", "plain", "none"])}
    heads, kv_heads, dim = rng.choice([(24, 4, 256), (32, 8, 128), (16, 16, 64), (14, 2, 128), (10, 1, 256),
                                       (8, 8, 128), (9, 3, 64)])
    new = _log_int(rng, 1, 2048)
    window = rng.choice([0, 0, 0, 1]) and _log_int(rng, 16, 4096)
    case = {"op": op, "requests": _log_int(rng, 1, 64), "new": new, "ctx": _log_int(rng, 1, 32768),
            "even": rng.random() < 0.5, "heads": heads, "kv_heads": kv_heads, "dim": dim,
            "page": rng.choice([16, 32, 64, 128]), "window": window,
            "sinks": rng.choice([0, 1, 4, 130]) if window else 0, "type": rng.choice(["bf16", "fp16"]),
            "lens_seed": rng.randrange(1 << 30)}
    while _too_large(case):
        big = "requests" if case["requests"] > 4 else "ctx" if case["ctx"] > case["new"] else "new"
        case[big] = max(1, case[big] * 2 // 3)
    return case


def _too_large(case):
    """Whether a drawn attention case's padded scores or keys would pass those of the largest listed ones."""
    pairs = case["requests"] * case["new"] * (case["ctx"] + case["new"]) * case["heads"]
    keys = case["requests"] * (case["ctx"] + case["new"]) * case["kv_heads"] * case["dim"]
    return pairs > 4.5e8 or pairs * case["dim"] > 1.1e11 or keys > 3.2e8


def _lengths(case):
    """Cached tokens and new tokens of each request: whole contexts of one order of size, or ragged ones."""
    g = np.random.default_rng(case["lens_seed"])
    r, ctx, new = case["requests"], case["ctx"], case["new"]
    lens = np.maximum(0, (ctx * g.uniform(0.5, 1.0, r)).astype(np.int64))
    if r == 1:
        lens[:] = ctx
    fresh = np.full(r, new) if case["even"] or new == 1 else np.maximum(1, (new * g.uniform(0.05, 1.0, r)).astype(np.int64))
    return lens, fresh


def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _int(values):
    return torch.as_tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    return {"tables": _prepare_tables, "append": _prepare_append, "attn": _prepare_attn,
            "sample": _prepare_sample}[case["op"]](case, seed)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"tables": _own_tables, "append": _own_append, "attn": _own_attn, "sample": _own_sample}[op](state)
    return {"tables": _plain_tables, "append": _plain_append, "attn": _plain_attn, "sample": _plain_sample}[op](state)


def exact(case, seed):
    return {"tables": _exact_tables, "append": _exact_append, "attn": _exact_attn,
            "sample": _exact_sample}[case["op"]](prepare(case, seed))


def work(case):
    op = case["op"]
    if op == "tables":
        lens, new = _lengths(case)
        r, page = case["requests"], case["page"]
        need = -(-(lens + new) // page) - -(-lens // page)
        return {"bytes": int(16 * r + 8 + 8 * need.sum() + 4 * r + 12 * new.sum()), "flops": 0}
    if op == "append":
        real = case["tokens"] - case["padding"] if case["tokens"] > case["padding"] else case["tokens"]
        return {"bytes": int(8 * case["tokens"] + 8 * real * case["kv_heads"] * case["dim"]), "flops": 0}
    if op == "sample":
        # the noise is read only where a token is kept, which the values decide: not counted
        n = case["rows"] * case["vocab"]
        return {"bytes": int(n * (4 if case["type"] == "fp32" else 2) + 20 * case["rows"]), "flops": 2 * n}
    lens, new = _lengths(case)
    keys = pairs = 0
    for old, n in zip(lens.tolist(), new.tolist()):
        p = np.arange(old, old + n)
        if case["window"]:
            near = np.minimum(p + 1, case["window"])
            first = np.minimum(p + 1 - near, case["sinks"])
            pairs += int((near + first).sum())
            low = max(0, old + 1 - case["window"])
            keys += old + n - low + min(low, case["sinks"])
        else:
            pairs += int((p + 1).sum())
            keys += old + n
    tokens = int(new.sum())
    return {"bytes": int(4 * keys * case["kv_heads"] * case["dim"] + 4 * tokens * case["heads"] * case["dim"]),
            "flops": int(4 * pairs * case["heads"] * case["dim"])}


# ---------------------------------------------------------------- page tables


def _prepare_tables(case, seed):
    lens, new = _lengths(case)
    # the lengths are the case's, their order among the requests the seed's
    order = np.random.default_rng(seed).permutation(len(lens))
    lens, new = lens[order], new[order]
    page, r = case["page"], case["requests"]
    owned = -(-lens // page)
    need = -(-(lens + new) // page) - owned
    max_blocks = int((owned + need).max()) + 2
    free = max(1, int(need.sum() * case["free"]))
    ids = np.random.default_rng(seed + 1).permutation(int(owned.sum()) + free).astype(np.int32)
    table = np.full((r, max_blocks), -1, np.int32)
    table[np.arange(max_blocks)[None] < owned[:, None]] = ids[free:]
    tokens = int(new.sum())
    out = (torch.empty(r + 1, dtype=torch.int32, device="cuda"), torch.empty(r, dtype=torch.int32, device="cuda"),
           torch.empty(tokens, dtype=torch.int32, device="cuda"), torch.empty(tokens, dtype=torch.int64, device="cuda"),
           torch.empty(3, dtype=torch.int32, device="cuda"))
    return {"case": case, "lens": _int(lens), "new": _int(new), "free": _int(ids[:free]), "num_free": _int([free]),
            "table": _int(table), "max_tokens": tokens, "out": out}


def _own_tables(s):
    from weight_only_groupwise_gb300 import nq
    out = nq.page_tables(s["lens"], s["new"], s["free"], s["num_free"], s["table"], s["case"]["page"],
                         s["max_tokens"], out=s["out"])
    return [s["table"], *out]


def _plain_tables(s):
    page, cap = s["case"]["page"], s["max_tokens"]
    old, n, table, free = s["lens"], s["new"], s["table"], s["free"]
    r, max_blocks = table.shape
    zero = torch.zeros(1, dtype=torch.int32, device=table.device)
    end = torch.cumsum(n.clamp(min=0), 0, dtype=torch.int32)
    q_start = torch.cat([zero, end]).clamp(max=cap)
    owned = (old + page - 1) // page
    valid = (old >= 0) & (n >= 0) & (old + n <= max_blocks * page) & (end <= cap)
    need = torch.where(valid, (old + n + page - 1) // page - owned, zero)
    upto = torch.cumsum(need, 0, dtype=torch.int32)
    admitted = valid & ((need == 0) | (upto <= s["num_free"]))
    j = torch.arange(max_blocks, device=table.device, dtype=torch.int32)[None]
    fresh = admitted[:, None] & (j >= owned[:, None]) & (j < (owned + need)[:, None])
    source = ((upto - need - owned)[:, None] + j).clamp(0, free.numel() - 1)
    table = torch.where(fresh, free[source.long()], table)
    t = torch.arange(cap, device=table.device, dtype=torch.int32)
    req = torch.searchsorted(q_start[1:], t, right=True).clamp(max=r - 1)
    pos = old[req] + t - q_start[req]
    live = admitted[req] & (t < q_start[-1])
    block = table[req, (pos // page).clamp(0, max_blocks - 1).long()]
    slots = torch.where(live, block.long() * page + pos % page, -1)
    taken = torch.where(admitted, need, zero).sum()
    counts = torch.stack([q_start[-1].long(), taken, (~admitted).sum()]).to(torch.int32)
    return [table, q_start, torch.where(admitted, old + n, zero), torch.where(live, pos, -1), slots, counts]


def _exact_tables(s):
    page, cap = s["case"]["page"], s["max_tokens"]
    old, n, free = (s[k].tolist() for k in ("lens", "new", "free"))
    table, left = s["table"].cpu().numpy().astype(np.int64), int(s["num_free"])
    q_start, kv, pos, slots = [0], [], [], []
    asked = taken = refused = 0
    for r, (a, m) in enumerate(zip(old, n)):
        have, want = -(-a // page), -(-(a + m) // page)
        first = q_start[-1]
        q_start.append(min(first + m, cap))
        ok = a + m <= table.shape[1] * page and first + m <= cap
        if ok:
            asked += want - have
            ok = want == have or asked <= left
        if not ok:
            refused += 1
            kv.append(0)
            pos += [-1] * (q_start[-1] - first)
            slots += [-1] * (q_start[-1] - first)
            continue
        table[r, have:want] = free[taken:taken + want - have]
        taken += want - have
        kv.append(a + m)
        pos += range(a, a + m)
        slots += [int(table[r, p // page]) * page + p % page for p in range(a, a + m)]
    pos += [-1] * (cap - len(pos))
    slots += [-1] * (cap - len(slots))
    return [torch.as_tensor(x).to(t) for x, t in
            ((table, torch.int32), (q_start, torch.int32), (kv, torch.int32), (pos, torch.int32),
             (slots, torch.int64), ([q_start[-1], taken, refused], torch.int32))]


# ---------------------------------------------------------------- KV append


def _prepare_append(case, seed):
    g, dtype = _rng(seed), DTYPES[case["type"]]
    t, h, d, page = case["tokens"], case["kv_heads"], case["dim"], case["page"]
    blocks = t // page * 2 + 9
    shape = (blocks, page, h, d)
    k = torch.randn((t, h, d), device="cuda", generator=g).to(dtype)
    v = torch.randn((t, h, d), device="cuda", generator=g).to(dtype)
    # whole pages in any order, as the page tables give them
    ids = torch.randperm(blocks, device="cuda", generator=g)[:t // page + 1]
    slots = (ids[:, None] * page + torch.arange(page, device="cuda")).reshape(-1)[:t].clone()
    if t > case["padding"] > 0:
        slots[t - case["padding"]:] = -1
    return {"case": case, "k": k, "v": v, "slots": slots,
            "k_cache": torch.randn(shape, device="cuda", generator=g).to(dtype),
            "v_cache": torch.randn(shape, device="cuda", generator=g).to(dtype)}


def _own_append(s):
    from weight_only_groupwise_gb300 import nq
    nq.kv_append(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
    return [s["k_cache"], s["v_cache"]]


def _plain_append(s):
    live = s["slots"] >= 0
    at = s["slots"][live]
    s["k_cache"].flatten(0, 1)[at] = s["k"][live]
    s["v_cache"].flatten(0, 1)[at] = s["v"][live]
    return [s["k_cache"], s["v_cache"]]


def _exact_append(s):
    out, slots = [], s["slots"].cpu().numpy()
    for new, cache in ((s["k"], s["k_cache"]), (s["v"], s["v_cache"])):
        rows = cache.cpu().double().numpy().reshape(-1, *new.shape[1:])
        rows[slots[slots >= 0]] = new.cpu().double().numpy()[slots >= 0]
        out.append(torch.from_numpy(rows.reshape(cache.shape)))
    return out


# ---------------------------------------------------------------- attention


def _prepare_attn(case, seed):
    g, dtype = _rng(seed), DTYPES[case["type"]]
    lens, new = _lengths(case)
    order = np.random.default_rng(seed).permutation(len(lens))
    lens, new = lens[order], new[order]
    total, page = lens + new, case["page"]
    blocks = -(-total // page)
    width, pool = int(blocks.max()) + 1, int(blocks.sum()) * 9 // 8 + 2
    ids = np.random.default_rng(seed + 1).permutation(pool).astype(np.int32)
    table = np.full((len(lens), width), -1, np.int32)
    table[np.arange(width)[None] < blocks[:, None]] = ids[:int(blocks.sum())]
    cache = (pool, page, case["kv_heads"], case["dim"])
    k = torch.randn(cache, device="cuda", generator=g, dtype=torch.float32).to(dtype)
    v = torch.randn(cache, device="cuda", generator=g, dtype=torch.float32).to(dtype)
    # queries of more than unit length: some tokens attend to few keys, some to many
    q = torch.randn((int(new.sum()), case["heads"], case["dim"]), device="cuda", generator=g)
    q = (q * torch.rand((q.shape[0], case["heads"], 1), device="cuda", generator=g).mul_(2.5).add_(0.5)).to(dtype)
    return {"case": case, "q": q, "k_cache": k, "v_cache": v, "table": _int(table),
            "q_start": _int(np.concatenate([[0], np.cumsum(new)])), "kv_lens": _int(total),
            "most_new": int(new.max()), "most_keys": int(total.max()), "scale": case["dim"] ** -0.5,
            "out": torch.empty_like(q)}


def _own_attn(s):
    from weight_only_groupwise_gb300 import nq
    case = s["case"]
    return nq.attn_paged(s["q"], s["k_cache"], s["v_cache"], s["table"], s["q_start"], s["kv_lens"],
                         scale=s["scale"], window=case["window"], sinks=case["sinks"], out=s["out"])


def _plain_attn(s):
    case, q, table = s["case"], s["q"], s["table"]
    heads, groups, dim, page = case["kv_heads"], case["heads"] // case["kv_heads"], case["dim"], case["page"]
    r, most, keys = table.shape[0], s["most_new"], s["most_keys"]
    j = torch.arange(keys, device=q.device)
    at = table[:, j // page].clamp(min=0).long() * page + j % page
    k = s["k_cache"].flatten(0, 1)[at].float().permute(0, 2, 3, 1)
    v = s["v_cache"].flatten(0, 1)[at].float().permute(0, 2, 1, 3)
    i = torch.arange(most, device=q.device)
    n = (s["q_start"][1:] - s["q_start"][:-1])[:, None]
    row = (s["q_start"][:-1, None] + i).clamp(max=q.shape[0] - 1).long()
    x = q[row].float().view(r, most, heads, groups, dim).permute(0, 2, 1, 3, 4).reshape(r, heads, -1, dim)
    scores = torch.matmul(x, k).mul_(s["scale"]).view(r, heads, most, groups, keys)
    pos = (s["kv_lens"][:, None] - n + i)[:, :, None]
    seen = (j <= pos) & (j < s["kv_lens"][:, None, None])
    if case["window"]:
        seen = seen & ((j > pos - case["window"]) | (j < case["sinks"]))
    hidden = ~seen[:, None, :, None, :]
    scores.masked_fill_(hidden, -math.inf)
    top = scores.amax(-1, keepdim=True).clamp(min=-3e38)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    o = torch.matmul(p.view(r, heads, -1, keys), v).view(r, heads, most, groups, dim)
    o = torch.where(total > 0, o / total, 0.0).permute(0, 2, 1, 3, 4).reshape(r, most, -1, dim)
    return o[i < n].to(q.dtype)


def _exact_attn(s):
    case, page = s["case"], s["case"]["page"]
    q, starts, kv, table = s["q"], s["q_start"].tolist(), s["kv_lens"].tolist(), s["table"]
    group = case["heads"] // case["kv_heads"]
    out = torch.zeros(q.shape, dtype=torch.float64, device=q.device)
    for r, end in enumerate(kv):
        a, b = starts[r], starts[r + 1]
        ids = table[r, :-(-end // page)].long()
        p = torch.arange(end - (b - a), end, device=q.device)[:, None]
        j = torch.arange(end, device=q.device)[None]
        seen = j <= p
        if case["window"]:
            seen &= (p - j < case["window"]) | (j < case["sinks"])
        for h in range(case["kv_heads"]):
            k = s["k_cache"][ids, :, h].reshape(-1, case["dim"])[:end].double()
            v = s["v_cache"][ids, :, h].reshape(-1, case["dim"])[:end].double()
            for g in range(h * group, h * group + group):
                w = torch.softmax((q[a:b, g].double() @ k.T * s["scale"]).masked_fill(~seen, -math.inf), -1)
                out[a:b, g] = w @ v
    return out


# ---------------------------------------------------------------- sampling


def _prepare_sample(case, seed):
    g = _rng(seed)
    rows, vocab = case["rows"], case["vocab"]
    # logits as a language model has them: a broad bulk, a few plausible tokens, some forbidden ones
    x = torch.randn((rows, vocab), device="cuda", generator=g) * 2.2
    hot = torch.randint(0, vocab, (rows, 40), device="cuda", generator=g)
    x.scatter_add_(1, hot, torch.rand((rows, 40), device="cuda", generator=g) * 12 + 2)
    off = torch.randint(0, vocab, (rows, vocab // 100), device="cuda", generator=g)
    x.scatter_(1, off, -math.inf)
    noise = torch.empty((rows, vocab), device="cuda").exponential_(generator=g)
    r = random.Random(seed)
    pick = {
        "usual": lambda: (0.7, 50, 0.9, 0.0),
        "plain": lambda: (1.0, 0, 1.0, 0.0),
        "none": lambda: (r.choice([0.3, 0.8, 1.0, 1.4]), 0, r.choice([0.5, 0.9, 0.99]), 0.0),
        "all": lambda: (r.choice([0.0, 0.5, 0.7, 1.0, 1.3]), r.choice([0, 1, 20, 50, 200, 5000]),
                        r.choice([1.0, 0.2, 0.8, 0.95, 0.99]), r.choice([0.0, 0.0, 0.02, 0.1])),
    }[case["mix"]]
    t, k, p, m = zip(*[pick() for _ in range(rows)])
    as_float = lambda a: torch.tensor(a, dtype=torch.float32, device="cuda")  # noqa: E731
    return {"case": case, "logits": x.to(DTYPES[case["type"]]), "noise": noise, "temperature": as_float(t),
            "top_k": _int(k), "top_p": as_float(p), "min_p": as_float(m),
            "out": torch.empty(rows, dtype=torch.int32, device="cuda")}


def _own_sample(s):
    from weight_only_groupwise_gb300 import nq
    return nq.sample(s["logits"], s["noise"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                     min_p=s["min_p"], out=s["out"])


def _plain_sample(s):
    x = torch.nan_to_num(s["logits"].float(), nan=-math.inf, posinf=math.inf, neginf=-math.inf)
    vocab = x.shape[1]
    t, k, p, least = (s[n][:, None] for n in ("temperature", "top_k", "top_p", "min_p"))
    x, order = torch.sort(x, dim=1, descending=True, stable=True)
    top = x[:, :1]
    d = torch.where(x == top, 0.0, (x - top) / t)
    rank = torch.arange(vocab, device=x.device)
    first = rank == 0
    kept = (x > -math.inf) & ((rank < k) | (k <= 0))
    w = torch.where(kept, torch.exp(d), 0.0)
    upto = torch.cumsum(w, 1)
    kept &= (upto - w < p * upto[:, -1:]) | (p >= 1)
    kept &= (d >= torch.log(least.clamp(max=1.0))) | (least <= 0)
    kept = torch.where(t > 0, kept, False) | first
    score = torch.where(kept, d - torch.log(s["noise"].gather(1, order)), -math.inf)
    best = kept & ((score == score.amax(1, keepdim=True)) | (t <= 0))
    token = torch.where(best, order, vocab).amin(1)
    return torch.where(top[:, 0] > -math.inf, token, -1).to(torch.int32)


def _exact_sample(s):
    x, noise = s["logits"].cpu().double().numpy(), s["noise"].cpu().double().numpy()
    settings = [s[n].cpu().double().tolist() for n in ("temperature", "top_k", "top_p", "min_p")]
    tokens = []
    for row, e, t, k, p, m in zip(x, noise, *settings):
        ids = np.lexsort((np.arange(row.size), -row))
        ids = ids[row[ids] > -np.inf]
        if not ids.size or t <= 0:
            tokens.append(int(ids[0]) if ids.size else -1)
            continue
        if k > 0:
            ids = ids[:int(k)]
        d = (row[ids] - row[ids[0]]) / t
        w = np.exp(d)
        n = ids.size
        if p < 1:
            n = max(1, int(np.searchsorted(np.concatenate([[0.0], np.cumsum(w)[:-1]]), p * w.sum())))
        if m > 0:
            n = max(1, min(n, int((d >= math.log(min(m, 1.0))).sum())))
        score = d[:n] - np.log(e[ids[:n]])
        tokens.append(int(ids[:n][score == score.max()].min()))
    return torch.tensor(tokens, dtype=torch.int32)
