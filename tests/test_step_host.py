"""The serving-step calls' argument checks: all run on the host, before any CUDA call, and return
the documented status. Fake device addresses are fine here. No GPU."""
import ctypes

import pytest

from weight_only_groupwise_gb300 import nq as nqmod

NULL, SHAPE, ALIGN, ALIAS, CUDA, DEVICE = -1, -2, -3, -4, -5, -6
A = 1 << 44          # fake device addresses this far apart
BF16, FP16, FP32 = 0, 1, 2


@pytest.fixture(scope="module")
def L():
    from weight_only_groupwise_gb300 import build
    build.build()
    return nqmod.lib()


def cache(K=A, V=2 * A, bs=64 * 4 * 256, rs=4 * 256, hs=256, blocks=100, page=64, heads=4, dim=256):
    return nqmod._KV.pack(K, V, bs, rs, hs, blocks, page, heads, dim)


def passes(status):
    """The checks let the call through: it ends at the missing GPU."""
    return status in (CUDA, DEVICE)


def gpu():
    import torch
    return torch.cuda.is_available()


def test_struct_matches_the_header(L):
    assert len(cache()) == 2 * ctypes.sizeof(ctypes.c_void_p) + 3 * 8 + 4 * 4


BAD_CACHES = [(dict(page=8), SHAPE), (dict(page=48), SHAPE), (dict(page=512), SHAPE), (dict(dim=96), SHAPE), (dict(heads=0), SHAPE),
              (dict(blocks=-1), SHAPE), (dict(rs=128), SHAPE), (dict(bs=1 << 38), SHAPE), (dict(K=0), NULL), (dict(V=0), NULL),
              (dict(K=A + 8), ALIGN), (dict(rs=4 * 256 + 4), ALIGN)]


def append(L, c=None, k=3 * A, ks=1024, v=4 * A, vs=1024, slots=5 * A, tokens=7):
    return L.nq_kv_append(k, ks, v, vs, slots, tokens, cache() if c is None else c, 0)


def attn(L, c=None, q=3 * A, qs=6144, table=4 * A, ts=50, blocks=50, q_start=5 * A, kv=6 * A, R=3, tokens=9, heads=24, scale=0.1,
         window=0, sinks=0, dtype=BF16, out=7 * A, os=6144):
    return L.nq_attn_paged(q, qs, cache() if c is None else c, table, ts, blocks, q_start, kv, R, tokens, heads, scale, window, sinks,
                           dtype, out, os, 0)


def tables(L, lens=A, new=2 * A, R=5, free=3 * A, cap=100, num=4 * A, page=64, table=5 * A, ts=30, blocks=30, q_start=6 * A, kv=7 * A,
           pos=8 * A, slots=9 * A, most=1000, counts=10 * A):
    return L.nq_page_tables(lens, new, R, free, cap, num, page, table, ts, blocks, q_start, kv, pos, slots, most, counts, 0)


def sample(L, logits=A, dtype=BF16, stride=1000, noise=2 * A, ns=1000, B=4, V=1000, t=3 * A, k=4 * A, p=5 * A, m=6 * A, tokens=7 * A):
    return L.nq_sample(logits, dtype, stride, noise, ns, B, V, t, k, p, m, tokens, 0)


@pytest.mark.parametrize("change,status", BAD_CACHES)
def test_caches(L, change, status):
    assert append(L, cache(**change)) == status
    assert attn(L, cache(**change)) == status


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), SHAPE), (dict(ks=1000), SHAPE), (dict(k=0), NULL), (dict(slots=0), NULL), (dict(v=4 * A + 2), ALIGN),
    (dict(ks=1028), ALIGN), (dict(slots=5 * A + 4), ALIGN), (dict(k=A + 1024), ALIAS), (dict(slots=2 * A), ALIAS)])
def test_append(L, change, status):
    assert append(L, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(tokens=-1), SHAPE), (dict(tokens=(1 << 23) + 1), SHAPE), (dict(R=-1), SHAPE), (dict(R=8193), SHAPE), (dict(ts=49), SHAPE),
    (dict(heads=6), SHAPE), (dict(heads=0), SHAPE), (dict(heads=4 * 129, qs=1 << 20, os=1 << 20), SHAPE), (dict(qs=6143), SHAPE),
    (dict(os=0), SHAPE), (dict(scale=0.0), SHAPE), (dict(scale=-1.0), SHAPE), (dict(scale=float("nan")), SHAPE),
    (dict(scale=float("inf")), SHAPE), (dict(window=-1), SHAPE), (dict(sinks=1), SHAPE), (dict(window=5, sinks=-1), SHAPE),
    (dict(dtype=FP32), SHAPE), (dict(dtype=-1), SHAPE), (dict(blocks=1 << 25, ts=1 << 25), SHAPE), (dict(q=0), NULL), (dict(out=0), NULL),
    (dict(table=0), NULL), (dict(q_start=0), NULL), (dict(kv=0), NULL), (dict(q=3 * A + 8), ALIGN), (dict(os=6148), ALIGN),
    (dict(kv=6 * A + 2), ALIGN), (dict(out=3 * A), ALIAS), (dict(out=A), ALIAS), (dict(out=2 * A + 16), ALIAS), (dict(out=4 * A), ALIAS),
    (dict(out=5 * A), ALIAS), (dict(out=6 * A), ALIAS)])
def test_attention(L, change, status):
    assert attn(L, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(R=-1), SHAPE), (dict(R=8193), SHAPE), (dict(page=24), SHAPE), (dict(cap=-1), SHAPE), (dict(ts=29), SHAPE), (dict(most=-1), SHAPE),
    (dict(R=0), SHAPE), (dict(lens=0), NULL), (dict(free=0), NULL), (dict(num=0), NULL), (dict(table=0), NULL), (dict(slots=0), NULL),
    (dict(counts=0), NULL), (dict(lens=A + 2), ALIGN), (dict(slots=9 * A + 4), ALIGN), (dict(kv=A), ALIAS), (dict(q_start=7 * A), ALIAS),
    (dict(pos=3 * A + 4), ALIAS), (dict(counts=5 * A + 16), ALIAS)])
def test_page_tables(L, change, status):
    assert tables(L, **change) == status


@pytest.mark.parametrize("change,status", [
    (dict(B=-1), SHAPE), (dict(V=0), SHAPE), (dict(V=524161, stride=1 << 20, ns=1 << 20), SHAPE), (dict(stride=999), SHAPE),
    (dict(ns=999), SHAPE), (dict(dtype=3), SHAPE), (dict(logits=0), NULL), (dict(noise=0), NULL), (dict(tokens=0), NULL),
    (dict(logits=A + 1), ALIGN), (dict(dtype=FP32, logits=A + 2), ALIGN), (dict(noise=2 * A + 2), ALIGN), (dict(tokens=A), ALIAS),
    (dict(tokens=2 * A + 64), ALIAS), (dict(tokens=5 * A), ALIAS)])
def test_sampling(L, change, status):
    assert sample(L, **change) == status


def test_empty_calls_are_accepted(L):
    assert append(L, tokens=0) == 0 and append(L, cache(K=0, V=0, blocks=0)) == 0
    assert attn(L, tokens=0) == 0
    assert tables(L, R=0, most=0) == 0
    assert sample(L, B=0) == 0


def test_good_calls_pass_the_checks(L):
    if gpu():
        pytest.skip("fake addresses: only where no GPU could be reached")
    assert passes(append(L)) and passes(attn(L)) and passes(tables(L)) and passes(sample(L))
    assert passes(sample(L, t=0, k=0, p=0, m=0)) and passes(attn(L, window=10, sinks=3, dtype=FP16))
    assert passes(L.nq_attn_reserve())
