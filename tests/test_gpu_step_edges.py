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
