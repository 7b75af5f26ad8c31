"""Plain 64-bit forms of the 8-bit products, and how far a result in 32 bits, rounded once, can be from them."""
import torch

E4M3 = torch.float8_e4m3fn


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def spread(s, K):
    """Scales [..][blocks] as one a column, for any block count."""
    return s.double().repeat_interleave(128, -1)[..., :K]


def activations(T, K, g, stride=None):
    """Random codes [T][K] (all 254 finite patterns) and scales; rows `stride` apart."""
    raw = torch.randint(0, 256, (T, stride or K), device="cuda", generator=g, dtype=torch.int32).to(torch.uint8)
    raw = torch.where((raw & 127) == 127, raw - 1, raw).view(E4M3)[:, :K]
    s = torch.exp(torch.randn((T, -(-K // 128)), device="cuda", generator=g)) * 2.0 ** -8
    return raw, s


def weights(E, N, K, g):
    c, _ = activations(E * N, K, g)
    s = torch.exp(torch.randn((E, -(-N // 128), -(-K // 128)), device="cuda", generator=g)) * 2.0 ** -8
    return c.reshape(E, N, K), s


def dense(c, s):
    """A weight [N][K] in 64 bits."""
    N, K = c.shape
    return c.double() * spread(s, K).repeat_interleave(128, 0)[:N]


def product(x, w):
    """(x w^T, how far a result of 32-bit sums can be from it): every product of two codes is exact; a block's sum of 128
    terms and the sum over blocks lose at most a last place (2^-23, for sums that are cut instead of rounded) an
    addition, the scales' product and the fused multiplication by it another two."""
    y = x @ w.T
    blocks = -(-x.shape[1] // 128)
    return y, (128 + blocks + 2) * 2.0 ** -23 * (x.abs() @ w.abs().T)


def silu(g, dg, u, du):
    """silu(g) u and its error: |silu'| < 1.1; the exponential's rounded argument loses |g| 2^-23 (two roundings of it), the
    exponential and the quotient two places each, sum and product a half."""
    s = g / (1 + torch.exp(-g))
    h = s * u
    return h, 1.1 * dg * (u.abs() + du) + s.abs() * du + (5 + g.abs()) * 2.0 ** -23 * h.abs()


def close(y, ref, err):
    """y, rounded once to its type (subnormals: half of the smallest), is within err of ref before that."""
    tiny = torch.finfo(y.dtype).smallest_normal * half_step(y.dtype)
    bound = err + half_step(y.dtype) * (ref.abs() + err) + tiny
    worst = ((y.double() - ref).abs() - bound).max()
    assert worst <= 0, f"off by {float(worst)} more than the bound {float(bound.max())}"


def close_codes(codes, scales, ref, err):
    """Codes and scales are those of values within err of ref."""
    N = ref.shape[1]
    pad = lambda t: torch.nn.functional.pad(t, (0, -N % 128)).view(t.shape[0], -1, 128)  # noqa: E731
    s_ref = pad(ref).abs().amax(-1) / 448
    ds = pad(err).amax(-1) / 448 + 2.0 ** -23 * s_ref + 2.0 ** -126
    assert bool(((scales.double() - s_ref).abs() <= ds).all())
    s = spread(scales, N)
    # e4m3: half a step is 2^-4 of the value, 2^-10 below the smallest normal number; the quotient loses a place
    step = s * torch.maximum(2.0 ** -4 * (ref.abs() + err) / s, torch.full_like(ref, 2.0 ** -10)) * (1 + 2.0 ** -19)
    # the block's largest value may land above 448 by the scale's own rounding, and is cut
    cut = 2.0 ** -22 * s * 448
    assert bool(((codes.double() * s - ref).abs() <= err + step + cut).all())


def quantised(x):
    """Codes and scales of x [rows][K] by the definition, in fp32."""
    rows, K = x.shape
    b = torch.nn.functional.pad(x.float(), (0, -K % 128)).view(rows, -1, 128)
    # (in 64 bits: division by a number is a multiplication by its rounded reciprocal on the GPU)
    s = (b.abs().amax(-1).double() / 448).float().clamp(min=2.0 ** -126)
    return (b / s[..., None]).clamp(-448, 448).to(E4M3).reshape(rows, -1)[:, :K], s
