"""The router and the combination against plain forms in 64 bits, and a layer of experts as it is used."""
import pytest
import torch

from tests import fp8_ref as ref
from weight_only_groupwise_gb300 import nq

pytestmark = pytest.mark.gpu
BF16, FP16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def built():
    from weight_only_groupwise_gb300 import build
    build.build()
    yield
    nq.device_error()


@pytest.fixture
def g(request):
    return torch.Generator(device="cuda").manual_seed(len(request.node.name))


def plain_route(logits, k, bias=None, score="softmax", normalize=True, scale=1.0):
    x = logits.double()
    x = torch.where(x.isnan(), -float("inf"), x)
    T, E = x.shape
    live = x > -float("inf")
    if score == "sigmoid":
        s = 1 / (1 + torch.exp(-x))
        if bias is not None:
            b = torch.where(bias.isnan(), -float("inf"), bias.double())
            live = live & (b > -float("inf"))
        key = x if bias is None else s + b
    else:
        top = x.amax(1, keepdim=True)
        s = torch.where(x == top, 1.0, torch.exp(x - top)) * live
        key = x
    key = torch.where(live, key, -float("inf"))
    order = torch.argsort(key, dim=1, descending=True, stable=True)[:, :k]
    kept = live.gather(1, order)
    chosen = torch.where(kept, s.gather(1, order), 0.0)
    if normalize:
        if score == "sigmoid":           # ratios of scores that 64 bits cannot hold either: from their logarithms
            log = torch.where(kept, torch.nn.functional.logsigmoid(x.gather(1, order)), -float("inf"))
            chosen = torch.where(kept, torch.exp(log - log.amax(1, keepdim=True)), 0.0)
        total = chosen.sum(1, keepdim=True)
        chosen = torch.where(total > 0, chosen / total, 0.0)
    elif score == "softmax":
        total = torch.where(live, s, 0.0).sum(1, keepdim=True)
        chosen = torch.where(total > 0, chosen / total, 0.0)
    ids = torch.where(kept, order, -1)
    return ids, chosen * scale


def check_route(logits, k, **how):
    T, E = logits.shape
    ids, weights, offsets, rows, slots = nq.moe_route(logits, k, **how)
    want, w = plain_route(logits, k, **how)
    assert torch.equal(ids.long(), want)
    # exp, the difference it is taken of, the sum of up to 1024 terms and the quotient: 2^-18 is 64 half places
    assert bool(((weights.double() - w).abs() <= 2.0 ** -18 * w + 1e-37).all())
    flat = ids.flatten().tolist()
    by = [[] for _ in range(E)]
    for i, e in enumerate(flat):
        if e >= 0:
            by[e].append(i)
    order = [i for b in by for i in b]
    ends = [0]
    for b in by:
        ends.append(ends[-1] + len(b))
    assert offsets.tolist() == ends
    assert rows.tolist() == [i // k for i in order] + [-1] * (T * k - len(order))
    where = [-1] * (T * k)
    for at, i in enumerate(order):
        where[i] = at
    assert slots.flatten().tolist() == where


@pytest.mark.parametrize("dtype", [BF16, FP16, F32])
@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 5, 5), (32, 128, 8), (33, 60, 4), (64, 256, 8), (257, 64, 6), (512, 32, 1), (513, 160, 6),
                                   (700, 500, 7), (100, 257, 32), (5000, 128, 8), (3000, 512, 3)])
def test_route(T, E, k, dtype, g):
    x = (2 * torch.randn((T, E), device="cuda", generator=g)).to(dtype)
    check_route(x, k)


@pytest.mark.parametrize("score,normalize,biased", [("softmax", False, False), ("sigmoid", True, False), ("sigmoid", False, False),
                                                   ("sigmoid", True, True), ("sigmoid", False, True)])
@pytest.mark.parametrize("T,E,k", [(40, 96, 8), (600, 256, 8)])
def test_route_scores(T, E, k, score, normalize, biased, g):
    x = 3 * torch.randn((T, E), device="cuda", generator=g)
    bias = 0.2 * torch.randn(E, device="cuda", generator=g) if biased else None
    check_route(x, k, score=score, normalize=normalize, bias=bias, scale=2.5)


def test_route_ties_go_to_the_lower_index(g):
    x = torch.randint(-2, 3, (300, 70), device="cuda", generator=g).float()
    x[x == 0] *= -1                      # both zeros are one value
    check_route(x, 9)
    check_route(torch.zeros((40, 33), device="cuda"), 4)
    # with a bias: equal inputs, and sums that only 64 bits tell apart
    check_route(x, 9, score="sigmoid", bias=torch.zeros(70, device="cuda"))
    near = 1 + 2.0 ** -22 * torch.randint(-8, 9, (64, 50), device="cuda", generator=g).float()
    check_route(near, 6, score="sigmoid", bias=0.3 + 2.0 ** -24 * torch.randint(-8, 9, (50,), device="cuda", generator=g).float())
    check_route(near, 6, score="sigmoid", bias=0.3 + 2.0 ** -24 * torch.randint(-8, 9, (50,), device="cuda", generator=g).float(), normalize=False)


@pytest.mark.parametrize("T", [37, 900])
def test_route_of_masked_and_unusual_rows(T, g):
    inf, nan = float("inf"), float("nan")
    x = 2 * torch.randn((T, 40), device="cuda", generator=g)
    x[2] = -inf
    x[3, 5:] = -inf
    x[4, ::2] = nan
    x[5] = nan
    x[6, 7] = inf
    x[7, 3:20] = inf
    x[8] = torch.finfo(F32).min
    x[9, 1:] = torch.finfo(F32).min
    x[20:] = -inf                        # padding
    check_route(x, 8)
    check_route(x, 8, normalize=False)
    bias = 0.1 * torch.randn(40, device="cuda", generator=g)
    check_route(x, 8, score="sigmoid", bias=bias)
    bias[3], bias[9] = -inf, nan
    check_route(x, 8, score="sigmoid", bias=bias)
    # scores far below zero keep their ratios
    check_route(x[10:20] - 300, 4, score="sigmoid")


def test_route_of_strided_rows_and_no_tokens(g):
    x = torch.randn((50, 200), device="cuda", generator=g)
    check_route(x[:, 3:77], 5)
    check_route(x.to(BF16)[:, 1:78], 5)
    _, _, offsets, _, _ = nq.moe_route(x[:0], 5)
    assert offsets.tolist() == [0] * 201


def plain_combine(y, slots, weights, base):
    live = (slots >= 0) & (slots < y.shape[0])
    rows = y.double()[slots.clamp(0, max(y.shape[0] - 1, 0)).long()]
    rows = torch.where(live[..., None], rows * weights.double()[..., None], 0.0)
    out, size = rows.sum(1), rows.abs().sum(1)
    if base is not None:
        out, size = out + base.double(), size + base.double().abs()
    return out, (slots.shape[1] + 1) * 2.0 ** -24 * size


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("T,k,N,base", [(1, 1, 8, False), (1, 8, 2048, True), (5, 3, 1032, True), (64, 32, 264, False), (1000, 6, 640, True)])
def test_combine(T, k, N, base, dtype, g):
    y = torch.randn((T * k + 3, N), device="cuda", generator=g).to(dtype)
    slots = torch.randint(-1, T * k + 4, (T, k), device="cuda", generator=g, dtype=torch.int32)
    w = torch.randn((T, k), device="cuda", generator=g)
    b = torch.randn((T, N), device="cuda", generator=g).to(dtype) if base else None
    out = nq.moe_combine(y, slots, w, base=b)
    ref.close(out, *plain_combine(y, slots, w, b))
    if base:
        assert nq.moe_combine(y, slots, w, base=b, out=b) is b and torch.equal(b, out)


def test_combine_skips_what_no_slot_names(g):
    y = torch.full((4, 16), float("nan"), device="cuda", dtype=BF16)
    slots = torch.tensor([[-1, 4], [1 << 30, -(1 << 31)]], dtype=torch.int32, device="cuda")
    w = torch.full((2, 2), float("nan"), device="cuda")
    assert bool((nq.moe_combine(y, slots, w) == 0).all())
    assert bool((nq.moe_combine(y[:0], slots, w) == 0).all())
    wide = torch.randn((6, 80), device="cuda", generator=g).to(BF16)
    out = torch.full((3, 64), 9.0, device="cuda", dtype=BF16)
    s = torch.tensor([[0, 5], [3, 3], [-1, 2]], dtype=torch.int32, device="cuda")
    w = torch.rand((3, 2), device="cuda", generator=g)
    nq.moe_combine(wide[:, 16:56], s, w, out=out[:, 8:48])
    ref.close(out[:, 8:48], *plain_combine(wide[:, 16:56], s, w, None))
    assert bool((out[:, :8] == 9).all()) and bool((out[:, 48:] == 9).all())


@pytest.mark.parametrize("T", [1, 20, 300])
def test_a_layer_of_experts(T, g):
    """Router, quantisation, the experts' SwiGLU and down products and the combination, against the layer in 64 bits on
    the same codes; as one captured graph, with padded tokens."""
    E, k, K, N = 24, 4, 512, 256
    x = torch.randn((T, K), device="cuda", generator=g).to(BF16)
    logits = torch.randn((T, E), device="cuda", generator=g)
    if T > 2:
        logits[T - 2:] = -float("inf")
    q = lambda E_, N_, K_: (lambda c, s: (c.view(E_, N_, K_), s))(  # noqa: E731
        (105 * torch.randn((E_ * N_, K_), device="cuda", generator=g)).clamp(-448, 448).to(ref.E4M3),
        torch.full((E_, -(-N_ // 128), -(-K_ // 128)), K_ ** -0.5 / 105, device="cuda"))
    wg, wu, wd = q(E, N, K), q(E, N, K), q(E, K, N)

    def layer():
        ids, weights, offsets, rows, slots = nq.moe_route(logits, k)
        codes, scales = nq.quant_fp8(x)
        h, hs = nq.swiglu_fp8_experts(codes, scales, *wg, *wu, offsets, rows=rows, dtype=ref.E4M3)
        y = nq.gemm_fp8_experts(h, hs, *wd, offsets)
        return nq.moe_combine(y, slots, weights, base=x), (ids, weights, offsets, rows, codes, scales, h, hs)

    out, (ids, weights, offsets, rows, codes, scales, h, hs) = layer()
    ends, a = offsets.tolist(), codes.double() * ref.spread(scales, K)
    y = torch.zeros((T * k, K), dtype=torch.float64, device="cuda")
    dy = torch.zeros_like(y)
    for e in range(E):
        r0, r1 = ends[e], ends[e + 1]
        if r0 < r1:
            part = a[rows[r0:r1].long()]
            ref.close_codes(h[r0:r1], hs[r0:r1], *ref.silu(*ref.product(part, ref.dense(wg[0][e], wg[1][e])),
                                                          *ref.product(part, ref.dense(wu[0][e], wu[1][e]))))
            y[r0:r1], dy[r0:r1] = ref.product(h[r0:r1].double() * ref.spread(hs[r0:r1], N), ref.dense(wd[0][e], wd[1][e]))
    slots = torch.full((T * k,), -1, dtype=torch.int64, device="cuda")
    order = torch.argsort(torch.where(ids >= 0, ids, E).flatten(), stable=True)[:ends[-1]]
    slots[order] = torch.arange(ends[-1], device="cuda")
    slots = slots.view(T, k)
    w = weights.double()[..., None]
    rows_of = lambda t: torch.where((slots >= 0)[..., None], t[slots.clamp(min=0)] * w, 0.0)  # noqa: E731
    want = x.double() + rows_of(y).sum(1)
    size = x.double().abs() + rows_of(y.abs()).sum(1)
    # the products are rounded to bf16 before they are combined
    err = rows_of(dy + 2.0 ** -8 * (y.abs() + dy)).sum(1) + (k + 1) * 2.0 ** -23 * size
    ref.close(out, want, err)
    if T > 2:
        assert torch.equal(out[T - 2:], x[T - 2:])
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured, _ = layer()
    for _ in range(2):
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(captured, out)
    # other inputs in the same buffers
    x.copy_(torch.randn((T, K), device="cuda", generator=g))
    logits[:max(T - 2, 1)].normal_(generator=g)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(captured, layer()[0])


def test_a_decoder_with_experts(capsys):
    """The example's decoder with layers of experts: the same prompts and draws twice give the same tokens."""
    from examples import serving_step as ex
    model = ex.Decoder(layers=2, hidden=512, heads=8, kv_heads=2, dim=64, inner=384, vocab=2048, experts=32, chosen=4)
    tokens = []
    for _ in range(2):
        draw = torch.Generator(device="cuda").manual_seed(5)
        prompts = [torch.randint(0, 2048, (n,), device="cuda", generator=draw) for n in (3, 70, 129)]
        server = ex.Server(model, 3, blocks=40, page=16, most_blocks=12)
        logits = server.prompt(prompts, 21)
        assert bool(logits.isfinite().all()) and float(logits.float().std()) > 0.1
        tokens.append(server.generate(logits, 6, draw, temperature=torch.tensor([0.0, 0.8, 1.0], device="cuda")))
        assert server.lens.tolist() == [9, 76, 135]
    assert torch.equal(*tokens) and int(tokens[0].min()) >= 0
    ex.main(16)
    assert "blocks left" in capsys.readouterr().out
