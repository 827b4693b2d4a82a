"""Plain binary64 forms of the feed-forward operators, on the CPU, from decoded operands (helpers
of the tests; nothing here uses the library)."""
import math

import torch

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0],
                    dtype=torch.float64)


def _e4m3_table():
    v = []
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        x = math.nan if (b & 127) == 127 else x
        v.append(-x if b > 127 else x)
    return torch.tensor(v, dtype=torch.float64)


E4M3 = _e4m3_table()


def nvfp4_values(codes, scales, s_enc):
    """[R, K] values of codes [R, K/2], scales [R, K/16] and s_enc (1 or R values)."""
    c = codes.cpu().long()
    v = torch.stack([E2M1[c & 15], E2M1[c >> 4]], 2).reshape(c.shape[0], 2 * c.shape[1])
    s = E4M3[scales.cpu().long()].repeat_interleave(16, 1)
    return v * s / s_enc.cpu().double().reshape(-1, 1)


def mxfp8_values(codes, scales, slab=False):
    c = codes.cpu().long()
    if slab:
        R, K = c.shape
        flat = c.reshape(-1)
        c = torch.cat([flat[b * K:min(R, b + 256) * K].reshape(K // 64, -1, 64).transpose(0, 1).reshape(-1, K)
                       for b in range(0, R, 256)])
    return E4M3[c] * torch.pow(2.0, scales.cpu().double() - 127).repeat_interleave(32, 1)


def act64(g, act):
    """(act(g), act'(g)); act 0 silu, 1 gelu, 2 gelu by tanh."""
    if act == 0:
        s = torch.sigmoid(g)
        return g * s, s + g * s * torch.sigmoid(-g)
    if act == 1:
        p = torch.special.erfc(-g / math.sqrt(2.0)) / 2
        return g * p, p + g * torch.exp(-g * g / 2) / math.sqrt(2 * math.pi)
    z = math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3)
    s = torch.sigmoid(z)
    return g * s, s + g * s * torch.sigmoid(-z) * math.sqrt(8 / math.pi) * (1 + 0.134145 * g * g)


# Bound of the device's activation against act64, relative to |act|: the exponential is exp2 of x log2 e, whose argument is rounded to 2^-24 of
# |x|; act matters only while it is above 2^-126, where |x| < 88, so e^x is within 88 2^-24 + a few 2^-24
# < 2^-17 of itself.  The erfc fit adds 2.1e-7 and x^2 its own 2^-24 x^2: the same 2^-17 covers it.
ACT_REL = 2.0 ** -17
F32 = 2.0 ** -24
BF16 = 2.0 ** -8


def act_rel(g, act):
    """Relative error of the device's act(g), and of each term of act'(g), in fp32: the exponential's argument
    z (g, g^2 / 2 or z(g)) carries at most 8 roundings, each worth |z| 2^-24 of the result; the exponential, the
    reciprocal and the products after it 10; the fit of the normal distribution function 2.1e-7 < 4 2^-24."""
    z = g.abs() if act == 0 else (g * g / 2 if act == 1 else math.sqrt(8 / math.pi) * (g + 0.044715 * g ** 3).abs())
    return (8 * z + 14) * F32


def act_grad_terms(g, act):
    """Sum of the magnitudes of act'(g)'s terms, which may cancel."""
    f, d = act64(g, act)
    s = torch.where(g == 0, torch.full_like(g, 0.5), f / torch.where(g == 0, torch.ones_like(g), g))
    return s.abs() + (d - s).abs()


def product(a, b):
    """(a b^T, sum |a b|) in binary64."""
    return a @ b.t(), a.abs() @ b.abs().t()


def sum_error(K, S, factors=2):
    """fp32 summation of K exact products in any order, plus `factors` roundings of the result."""
    return (K + factors) * F32 * S


def gated_error(g, u, eg, eu, act):
    """First-order error of act(g) u for g, u off by eg, eu (|act'| <= 1.13), before h's own rounding."""
    f, _ = act64(g, act)
    return 1.13 * eg * (u.abs() + eu) + f.abs() * eu + (f * u).abs() * (ACT_REL + 4 * F32)


def store_error(v, dtype):
    """Half a step of the stored type (and its smallest subnormal's half below the normal range)."""
    return v.abs() * BF16 + 2.0 ** -134 if dtype == torch.bfloat16 else v.abs() * F32 + 2.0 ** -150


def assert_within(got, want, tol, what):
    got = got.detach().cpu().double()
    assert got.shape == want.shape, (what, got.shape, want.shape)
    assert torch.equal(torch.isnan(got), torch.isnan(want)), what + ": NaN in other places"
    fin = torch.isfinite(want)
    assert torch.equal(got[~fin & ~torch.isnan(want)], want[~fin & ~torch.isnan(want)]), what + ": infinities differ"
    d = (got - want).abs()
    bad = fin & ~(d <= tol)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError("%s: %d of %d outside; first at %s: got %r want %r tol %r"
                             % (what, int(bad.sum()), bad.numel(), i, got[i].item(), want[i].item(), tol[i].item()))
