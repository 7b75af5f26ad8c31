"""What is measured of the 8-bit products and the experts' layer: quantisation of activations, block-scaled
matrix products and SwiGLU blocks, the router, the experts' ragged products and their combination.

A layer of experts takes them in the order route, quantise, SwiGLU of the experts, their down projection, combine; a
dense one quantise, SwiGLU, product. `run` makes the framework's calls where `own` is true, else the same results
from elementary torch operations in 32 bits. Sizes are this repository's 27B-class layer (hidden 5120, inner 17408)
or generic.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32, "e4m3": torch.float8_e4m3fn}
BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "e4m3": 1}
BLOCK = 128


def listed():
    return [
        # the activations of a verify batch before an 8-bit product
        {"name": "quant_verify", "op": "quant", "rows": 64, "K": 5120, "type": "bf16"},
        # a long prompt chunk's inner activations
        {"name": "quant_prompt", "op": "quant", "rows": 8191, "K": 17408, "type": "fp16"},
        # a verify batch's product: the weights' bytes
        {"name": "gemm_verify", "op": "gemm", "T": 16, "K": 5120, "N": 17408, "glu": False, "type": "bf16"},
        # a short prompt, sizes that fill no tile
        {"name": "gemm_odd", "op": "gemm", "T": 333, "K": 4112, "N": 2501, "glu": False, "type": "fp16"},
        # a prompt chunk's SwiGLU block, its result quantised for the down projection: the compute-bound end
        {"name": "swiglu_prompt", "op": "gemm", "T": 2048, "K": 5120, "N": 17408, "glu": True, "type": "e4m3"},
        # a decode step of a batch
        {"name": "route_decode", "op": "route", "T": 32, "E": 128, "k": 8, "score": "softmax", "normalize": True,
         "scale": 1.0, "bias": False, "padding": 0, "type": "bf16"},
        # prompt chunks, padded as for a captured graph, selection by biased scores
        {"name": "route_prompt", "op": "route", "T": 16384, "E": 256, "k": 8, "score": "sigmoid", "normalize": True,
         "scale": 2.5, "bias": True, "padding": 300, "type": "fp32"},
        # a decode step of a batch through many small experts: their weights' bytes
        {"name": "experts_decode", "op": "experts", "T": 32, "k": 8, "E": 128, "K": 2048, "N": 768, "glu": True,
         "gather": True, "type": "e4m3", "skew": 0.5, "lens_seed": 1},
        # a prompt chunk through large experts of uneven popularity
        {"name": "experts_prompt", "op": "experts", "T": 4096, "k": 8, "E": 64, "K": 4096, "N": 1408, "glu": True,
         "gather": True, "type": "e4m3", "skew": 0.5, "lens_seed": 2},
        # the small experts' down projection for a prompt chunk
        {"name": "experts_down", "op": "experts", "T": 4095, "k": 6, "E": 128, "K": 768, "N": 2048, "glu": False,
         "gather": False, "type": "bf16", "skew": 0.5, "lens_seed": 3},
        # a decode step's results
        {"name": "combine_decode", "op": "combine", "T": 32, "k": 8, "N": 2048, "base": True, "padding": 0, "type": "bf16"},
        # a prompt chunk's, added to a shared expert's
        {"name": "combine_prompt", "op": "combine", "T": 8192, "k": 8, "N": 4096, "base": True, "padding": 100,
         "type": "bf16"},
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(max(lo, hi))))))


def draw(rng):
    op = rng.choice(["quant", "gemm", "gemm", "gemm", "route", "experts", "experts", "experts", "combine"])
    if op == "quant":
        rows = _log_int(rng, 1, 8191)
        return {"op": op, "rows": rows, "K": 16 * _log_int(rng, 1, min(1280, 8191 * 1088 // rows)),
                "type": rng.choice(["bf16", "fp16", "fp32"]) if rows < 4000 else rng.choice(["bf16", "fp16"])}
    if op == "gemm":
        glu = rng.random() < 0.4
        case = {"op": op, "T": _log_int(rng, 1, 4096), "K": 16 * _log_int(rng, 8, 1088),
                "N": 16 * _log_int(rng, 4, 1088) if glu or rng.random() < 0.7 else _log_int(rng, 50, 17000), "glu": glu,
                "type": rng.choice(["bf16", "fp16", "e4m3"] if glu else ["bf16", "fp16"])}
        while work(case)["flops"] > 7.2e11:
            case["T"] = max(1, case["T"] * 2 // 3)
        return case
    if op == "route":
        E = _log_int(rng, 4, 500)
        score = rng.choice(["softmax", "sigmoid"])
        T = _log_int(rng, 1, min(16384, 16384 * 256 // E))
        return {"op": op, "T": T, "E": E, "k": min(E, _log_int(rng, 1, 12)), "score": score,
                "normalize": rng.random() < 0.7, "scale": rng.choice([1.0, 2.5]),
                "bias": score == "sigmoid" and rng.random() < 0.5, "padding": rng.choice([0, 0, min(T - 1, 17)]),
                "type": rng.choice(["bf16", "fp16", "fp32"])}
    if op == "experts":
        glu = rng.random() < 0.5
        E = _log_int(rng, 3, 200)
        case = {"op": op, "T": _log_int(rng, 1, 4096), "k": min(E, _log_int(rng, 1, 8)), "E": E,
                "K": 16 * _log_int(rng, 16, 320), "N": 16 * _log_int(rng, 8, 200) if glu else _log_int(rng, 128, 4500),
                "glu": glu, "gather": rng.random() < 0.6, "type": rng.choice(["bf16", "fp16", "e4m3"] if glu else ["bf16", "fp16"]),
                "skew": rng.choice([0.0, 0.5, 1.0]), "lens_seed": rng.randrange(1 << 30)}
        while case["E"] * case["K"] * case["N"] * (1 + glu) > 7e8:
            case["K"] = max(256, case["K"] * 2 // 3 // 16 * 16)
            case["N"] = max(128, case["N"] * 2 // 3 // 16 * 16)
        while 2 * case["T"] * case["k"] * case["K"] * case["N"] * (1 + glu) > 7.2e11:
            case["T"] = max(1, case["T"] * 2 // 3)
        return case
    T = _log_int(rng, 1, 8192)
    return {"op": op, "T": T, "k": _log_int(rng, 1, 8), "N": 8 * _log_int(rng, 16, min(1024, 8192 * 512 // T)),
            "base": rng.random() < 0.6, "padding": rng.choice([0, 0, min(T - 1, 9)]), "type": rng.choice(["bf16", "fp16"])}


def _routing(case):
    """[tokens][k]: distinct experts of each token, some experts more popular than others; the sizes of
    the experts' groups are the case's."""
    g = np.random.default_rng(case["lens_seed"])
    liking = case["skew"] * g.standard_normal(case["E"]).astype(np.float32)
    noise = g.gumbel(size=(case["T"], case["E"])).astype(np.float32)
    return np.argpartition(-(liking + noise), case["k"] - 1, axis=1)[:, :case["k"]]


def _rng(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return g


def _int(values):
    return torch.as_tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def prepare(case, seed):
    return {"quant": _prepare_quant, "gemm": _prepare_gemm, "route": _prepare_route, "experts": _prepare_experts,
            "combine": _prepare_combine}[case["op"]](case, seed)


def run(state):
    op = state["case"]["op"]
    if own:
        return {"quant": _own_quant, "gemm": _own_gemm, "route": _own_route, "experts": _own_experts,
                "combine": _own_combine}[op](state)
    return {"quant": _plain_quant, "gemm": _plain_gemm, "route": _plain_route, "experts": _plain_experts,
            "combine": _plain_combine}[op](state)


def exact(case, seed):
    return {"quant": _exact_quant, "gemm": _exact_gemm, "route": _exact_route, "experts": _exact_experts,
            "combine": _exact_combine}[case["op"]](prepare(case, seed))


def work(case):
    op = case["op"]
    if op == "quant":
        n = case["rows"] * case["K"]
        return {"bytes": int(n * (BYTES[case["type"]] + 1) + 4 * case["rows"] * -(-case["K"] // BLOCK)), "flops": 2 * n}
    if op == "route":
        T, k = case["T"], case["k"]
        return {"bytes": int(T * case["E"] * BYTES[case["type"]] + 16 * T * k + 4 * case["E"] * (2 if case["bias"] else 1)),
                "flops": 4 * T * case["E"]}
    if op == "combine":
        T, k, live = case["T"], case["k"], case["T"] - case["padding"]
        return {"bytes": int(2 * case["N"] * (live * k + T * (2 if case["base"] else 1)) + 8 * T * k),
                "flops": 2 * live * k * case["N"]}
    K, N, both = case["K"], case["N"], 2 if case["glu"] else 1
    blocks = -(-K // BLOCK)
    weight = both * (N * K + 4 * -(-N // BLOCK) * blocks)
    out = N * BYTES[case["type"]] + (4 * -(-N // BLOCK) if case["type"] == "e4m3" else 0)
    if op == "gemm":
        return {"bytes": int(weight + case["T"] * (K + 4 * blocks + out)), "flops": 2 * both * case["T"] * K * N}
    ids = _routing(case)
    rows, used = ids.size, np.unique(ids).size
    x_rows = case["T"] if case["gather"] else rows
    return {"bytes": int(used * weight + x_rows * (K + 4 * blocks) + rows * (out + (4 if case["gather"] else 0)) + 4 * case["E"]),
            "flops": 2 * both * rows * K * N}


# ---------------------------------------------------------------- codes and scales


def _blocks(x):
    """[rows][K] as [rows][blocks][128], zeros behind a last short block."""
    rows, K = x.shape
    return torch.nn.functional.pad(x, (0, -K % BLOCK)).view(rows, -1, BLOCK)


def _quantised(x):
    """fp32 [rows][K] -> (e4m3 codes, fp32 scales): a scale for each 128 columns of a row."""
    b = _blocks(x)
    s = (b.abs().amax(-1) / 448).clamp(min=2.0 ** -126)
    c = (b / s[..., None]).clamp(-448, 448).to(torch.float8_e4m3fn)
    return c.reshape(x.shape[0], -1)[:, :x.shape[1]].contiguous(), s


def _spread(s, K):
    """Scales [..][blocks] as one a column."""
    return s.repeat_interleave(BLOCK, -1)[..., :K]


def _weight(g, E, N, K):
    """Codes [E][N][K] and scales [E][N/128][K/128] of weights whose blocks differ in size."""
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    # a normal block's largest of 16384 values is about 4.2 of them
    codes = torch.randn((E, N, K), device="cuda", generator=g).mul_(105).clamp_(-448, 448).to(torch.float8_e4m3fn)
    s = torch.exp(0.4 * torch.randn((E, nb, kb), device="cuda", generator=g)) * (K ** -0.5 / 105)
    return codes, s


def _rows(g, T, K):
    """Activations: a few channels much larger than the others, tokens of different size."""
    x = torch.randn((T, K), device="cuda", generator=g) * torch.exp(0.5 * torch.randn((T, 1), device="cuda", generator=g))
    return x * (1 + 15 * (torch.rand((1, K), device="cuda", generator=g) < 0.004))


def _prepare_quant(case, seed):
    return {"case": case, "x": _rows(_rng(seed), case["rows"], case["K"]).to(DTYPES[case["type"]])}


def _own_quant(s):
    from weight_only_groupwise_gb300 import nq
    return list(nq.quant_fp8(s["x"]))


def _plain_quant(s):
    return list(_quantised(s["x"].float()))


def _exact_quant(s):
    x = s["x"].double()
    codes, scales = [], []
    for a in range(0, x.shape[1], BLOCK):
        part = x[:, a:a + BLOCK]
        scale = torch.clamp(part.abs().amax(1, keepdim=True) / 448, min=2.0 ** -126)
        # codes belong to the 32-bit scale that is stored with them
        codes.append((part / scale.float().double()).clamp(-448, 448).float().to(torch.float8_e4m3fn).double())
        scales.append(scale)
    return [torch.cat(codes, 1), torch.cat(scales, 1)]


# ---------------------------------------------------------------- products


def _prepare_gemm(case, seed):
    g = _rng(seed)
    T, K, N = case["T"], case["K"], case["N"]
    x, xs = _quantised(_rows(g, T, K))
    weights = [_weight(g, 1, N, K) for _ in range(2 if case["glu"] else 1)]
    return {"case": case, "x": x, "xs": xs, "w": [(c[0], s[0]) for c, s in weights]}


def _own_gemm(s):
    from weight_only_groupwise_gb300 import nq
    dtype = DTYPES[s["case"]["type"]]
    if s["case"]["glu"]:
        y = nq.swiglu_fp8(s["x"], s["xs"], *s["w"][0], *s["w"][1], dtype=dtype)
        return list(y) if isinstance(y, tuple) else [y]
    return [nq.gemm_fp8(s["x"], s["xs"], *s["w"][0], dtype=dtype)]


def _dequantised(codes, scales):
    """fp32 weights [E][N][K]."""
    N, K = codes.shape[-2:]
    return codes.float().mul_(_spread(scales, K).repeat_interleave(BLOCK, -2)[..., :N, :])


def _finish(parts, dtype):
    y = parts[0] if len(parts) == 1 else parts[0] * torch.sigmoid(parts[0]) * parts[1]
    return list(_quantised(y)) if dtype == torch.float8_e4m3fn else [y.to(dtype)]


def _plain_gemm(s):
    x = s["x"].float() * _spread(s["xs"], s["case"]["K"])
    return _finish([x @ _dequantised(c, sc).T for c, sc in s["w"]], DTYPES[s["case"]["type"]])


def _exact_rows(x, xs, weights, dtype):
    """The products of some rows with one expert's weights in 64 bits, finished as the case says."""
    K = x.shape[1]
    col = torch.arange(K, device=x.device) // BLOCK
    a = x.double() * xs.double()[:, col]
    parts = []
    for c, sc in weights:
        row = torch.arange(c.shape[0], device=x.device) // BLOCK
        parts.append(a @ (c.double() * sc.double()[row][:, col]).T)
    y = parts[0] if len(parts) == 1 else parts[0] / (1 + torch.exp(-parts[0])) * parts[1]
    if dtype != torch.float8_e4m3fn:
        return [y]
    return _exact_quant({"x": y})


def _exact_gemm(s):
    return _exact_rows(s["x"], s["xs"], s["w"], DTYPES[s["case"]["type"]])


# ---------------------------------------------------------------- router


def _prepare_route(case, seed):
    g = _rng(seed)
    T, E = case["T"], case["E"]
    x = 1.5 * torch.randn((T, E), device="cuda", generator=g) + torch.randn((1, E), device="cuda", generator=g)
    # padded rows choose no expert
    if case["padding"]:
        x[T - case["padding"]:] = -math.inf
    bias = 0.1 * torch.randn(E, device="cuda", generator=g) if case["bias"] else None
    return {"case": case, "logits": x.to(DTYPES[case["type"]]), "bias": bias}


def _own_route(s):
    from weight_only_groupwise_gb300 import nq
    case = s["case"]
    return list(nq.moe_route(s["logits"], case["k"], bias=s["bias"], score=case["score"], normalize=case["normalize"],
                             scale=case["scale"]))


def _plain_route(s):
    case = s["case"]
    T, E, k = case["T"], case["E"], case["k"]
    x = s["logits"].double()
    score = torch.sigmoid(x) if case["score"] == "sigmoid" else torch.exp(x - x.amax(1, keepdim=True).clamp(min=-1e300))
    key = x if s["bias"] is None else torch.where(x > -math.inf, score + s["bias"].double(), -math.inf)
    key, order = torch.sort(key, dim=1, descending=True, stable=True)
    ids = torch.where(key[:, :k] > -math.inf, order[:, :k], -1)
    chosen = torch.where(ids >= 0, score.gather(1, ids.clamp(min=0)), 0.0)
    if case["normalize"]:
        chosen = chosen / chosen.sum(1, keepdim=True).clamp(min=1e-300)
    elif case["score"] == "softmax":
        chosen = chosen / score.sum(1, keepdim=True).clamp(min=1e-300)
    weights = (chosen * case["scale"]).float()
    expert = torch.where(ids >= 0, ids, E).flatten()
    by_expert, place = torch.sort(expert, stable=True)
    offsets = torch.searchsorted(by_expert, torch.arange(E + 1, device=x.device))
    rows = torch.where(by_expert < E, place // k, -1)
    slots = torch.empty_like(place)
    slots[place] = torch.where(by_expert < E, torch.arange(T * k, device=x.device), -1)
    i32 = torch.int32
    return [ids.to(i32), weights, offsets.to(i32), rows.to(i32), slots.view(T, k).to(i32)]


def _exact_route(s):
    case = s["case"]
    E, k = case["E"], case["k"]
    x = s["logits"].cpu().double().numpy()
    bias = np.zeros(E) if s["bias"] is None else s["bias"].cpu().double().numpy()
    live = x > -np.inf
    with np.errstate(invalid="ignore"):
        if case["score"] == "sigmoid":
            score = 1 / (1 + np.exp(-x))
            key = x if s["bias"] is None else np.where(live, score + bias, -np.inf)
        else:
            score = np.where(live, np.exp(x - x.max(1, keepdims=True)), 0.0)
            key = x
    order = np.argsort(-key, axis=1, kind="stable")[:, :k]
    kept = np.take_along_axis(live, order, 1)
    chosen = np.where(kept, np.take_along_axis(score, order, 1), 0.0)
    if case["normalize"] or case["score"] == "softmax":
        total = chosen.sum(1, keepdims=True) if case["normalize"] else score.sum(1, keepdims=True)
        chosen = np.divide(chosen, total, out=np.zeros_like(chosen), where=total > 0)
    ids = np.where(kept, order, -1)
    rows, slots, offsets = np.full(ids.size, -1), np.full(ids.shape, -1), [0]
    for e in range(E):
        token, j = np.nonzero(ids == e)
        at = offsets[-1] + np.arange(token.size)
        rows[at], slots[token, j] = token, at
        offsets.append(offsets[-1] + token.size)
    as_int = lambda v: torch.as_tensor(np.asarray(v), dtype=torch.int32)  # noqa: E731
    return [as_int(ids), torch.from_numpy(chosen * case["scale"]), as_int(offsets), as_int(rows), as_int(slots)]


# ---------------------------------------------------------------- experts


def _prepare_experts(case, seed):
    g = _rng(seed)
    T, k, E, K, N = (case[n] for n in ("T", "k", "E", "K", "N"))
    ids = _routing(case)[np.random.default_rng(seed).permutation(T)]
    order = np.argsort(ids.reshape(-1), kind="stable")
    sizes = np.bincount(ids.reshape(-1), minlength=E)
    x, xs = _quantised(_rows(g, T if case["gather"] else T * k, K))
    return {"case": case, "x": x, "xs": xs, "w": [_weight(g, E, N, K) for _ in range(2 if case["glu"] else 1)],
            "offsets": _int(np.concatenate([[0], np.cumsum(sizes)])),
            "rows": _int(order // k) if case["gather"] else None, "most": int(sizes.max())}


def _own_experts(s):
    from weight_only_groupwise_gb300 import nq
    dtype = DTYPES[s["case"]["type"]]
    if s["case"]["glu"]:
        y = nq.swiglu_fp8_experts(s["x"], s["xs"], *s["w"][0], *s["w"][1], s["offsets"], rows=s["rows"], dtype=dtype)
        return list(y) if isinstance(y, tuple) else [y]
    return [nq.gemm_fp8_experts(s["x"], s["xs"], *s["w"][0], s["offsets"], rows=s["rows"], dtype=dtype)]


def _plain_experts(s):
    case = s["case"]
    K, M = case["K"], case["T"] * case["k"]
    x = s["x"].float() * _spread(s["xs"], K)
    if s["rows"] is not None:
        x = x[s["rows"].long()]
    i = torch.arange(M, device=x.device)
    expert = torch.searchsorted(s["offsets"][1:].long(), i, right=True)
    at = expert * s["most"] + i - s["offsets"][expert]
    padded = x.new_zeros((case["E"] * s["most"], K))
    padded[at] = x
    padded = padded.view(case["E"], s["most"], K)
    return _finish([torch.bmm(padded, _dequantised(c, sc).mT).flatten(0, 1)[at] for c, sc in s["w"]],
                   DTYPES[case["type"]])


def _exact_experts(s):
    case, ends = s["case"], s["offsets"].tolist()
    rows = None if s["rows"] is None else s["rows"].long()
    parts = []
    for e in range(case["E"]):
        a, b = ends[e], ends[e + 1]
        if a == b:
            continue
        pick = slice(a, b) if rows is None else rows[a:b]
        parts.append(_exact_rows(s["x"][pick], s["xs"][pick], [(c[e], sc[e]) for c, sc in s["w"]], DTYPES[case["type"]]))
    return [torch.cat(p) for p in zip(*parts)]


# ---------------------------------------------------------------- combination


def _prepare_combine(case, seed):
    g, dtype = _rng(seed), DTYPES[case["type"]]
    T, k, N, live = case["T"], case["k"], case["N"], case["T"] - case["padding"]
    # the rows lie in the order of their experts: anywhere; padded tokens have none
    slots = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    slots[:live] = torch.randperm(live * k, device="cuda", generator=g).view(live, k).to(torch.int32)
    weights = torch.rand((T, k), device="cuda", generator=g) + 0.05
    return {"case": case, "y": torch.randn((live * k, N), device="cuda", generator=g).to(dtype), "slots": slots,
            "weights": weights / weights.sum(1, keepdim=True),
            "base": torch.randn((T, N), device="cuda", generator=g).to(dtype) if case["base"] else None}


def _own_combine(s):
    from weight_only_groupwise_gb300 import nq
    return [nq.moe_combine(s["y"], s["slots"], s["weights"], base=s["base"])]


def _plain_combine(s):
    w = torch.where(s["slots"] >= 0, s["weights"], 0.0)
    y = (s["y"].float()[s["slots"].clamp(min=0).long()] * w[..., None]).sum(1)
    if s["base"] is not None:
        y = y + s["base"].float()
    return [y.to(s["y"].dtype)]


def _exact_combine(s):
    T, k = s["slots"].shape
    y = torch.zeros((T, s["y"].shape[1]), dtype=torch.float64, device=s["y"].device)
    if s["base"] is not None:
        y += s["base"].double()
    for j in range(k):
        at = s["slots"][:, j].long()
        live = at >= 0
        y[live] += s["weights"][live, j, None].double() * s["y"][at[live]].double()
    return [y]
