"""The serving-step calls together, as examples/serving_step.py makes them."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ex():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    from weight_only_groupwise_gb300 import build
    build.build()
    from examples import serving_step
    return serving_step


def test_a_prompts_chunks_do_not_matter(ex):
    """The same prompts in chunks of different sizes give the same logits, up to what a bf16
    rounding of the activations (2^-8) does over two layers, and generation follows on."""
    model = ex.Decoder(layers=2, hidden=512, heads=8, kv_heads=2, dim=64, inner=1024, vocab=4096)
    g = torch.Generator(device="cuda").manual_seed(2)
    prompts = [torch.randint(0, 4096, (n,), device="cuda", generator=g) for n in (3, 70, 129)]
    got = []
    for chunk in (21, 8, 1):
        server = ex.Server(model, 3, blocks=40, page=16, most_blocks=12)
        got.append(server.prompt(prompts, chunk).double())
        assert server.lens.tolist() == [3, 70, 129]
        owned = [server.table[r, :-(-n // 16)].tolist() for r, n in enumerate((3, 70, 129))]
        ids = sum(owned, [])
        assert len(set(ids)) == len(ids) == 40 - int(server.num_free) and int(server.refused) == 0
    for other in got[1:]:
        assert ((other - got[0]).norm() / got[0].norm()).item() < 0.03
    tokens = server.generate(got[-1].to(torch.bfloat16), 5, g, temperature=torch.tensor([0.0, 0.8, 1.0], device="cuda"),
                             top_p=torch.tensor([1.0, 0.9, 0.95], device="cuda"))
    assert tokens.shape == (3, 5) and int(tokens.min()) >= 0 and int(tokens.max()) < 4096
    assert server.lens.tolist() == [8, 75, 134]
    assert tokens[0, 0].item() == int(got[-1][0].argmax())


def test_main_runs(ex, capsys):
    ex.main()
    assert "blocks left" in capsys.readouterr().out


@pytest.mark.parametrize("new,dim,heads", [([1, 2, 8], 128, 8), ([700, 200], 256, 24)])
def test_a_wait_that_runs_out_is_reported_and_the_next_call_is_right(ex, new, dim, heads):
    """As for the projections: a bound of 1 ns makes the attention blocks (and pairs of blocks) abort."""
    from tests import gpu_util as gu
    from tests.test_gpu_attn import problem, reference
    nq = ex.nq
    p = problem([3000] * len(new), new, heads, heads // 4 if dim == 128 else 4, dim, 64, torch.bfloat16, seed=dim)
    call = lambda: nq.attn_paged(p["q"], p["k"], p["v"], p["table"], p["q_start"], p["kv"])  # noqa: E731
    gu.expect_timeout(nq, call)
    out = call()
    nq.device_error()
    ref, bound = reference(p, dim ** -0.5)
    assert ((out.double() - ref).abs() <= bound).all()
