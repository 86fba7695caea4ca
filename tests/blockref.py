"""Definitions of the E4M3 operators with a scale for each block of 128, for the tests.

Bounds.  A product passes at most 128 additions in its block, G over the blocks and 8 where parts of K meet, and two
scalings; each loses at most 2^-23 of the sum of magnitudes A (2^-24 where it rounds, 2^-23 where it cuts off):
(140 + G) 2^-23 A."""
import torch

F8 = torch.float8_e4m3fn


def quantise(v, amax):
    """Codes of fp32 values [..., 128] whose block has the maximum amax [...], and the scale: IEEE quotients."""
    s = amax / 448.0
    by = torch.where(s > 0, s, torch.ones_like(s))[..., None]
    return torch.where(s[..., None] > 0, (v / by).clamp(-448.0, 448.0), torch.zeros_like(v)).to(F8), s


def act_codes(x):
    """x [M][K] -> (uint8 [M][K], fp32 [K / 128][M]), on the CPU."""
    M, K = x.shape
    v = x.cpu().float().view(M, K // 128, 128)
    c, s = quantise(v, v.abs().amax(-1))
    return c.view(torch.uint8).view(M, K), s.t().contiguous()


def weight_codes(w):
    """w [N][K] -> (uint8 [N][K], fp32 [ceil(N / 128)][K / 128]), on the CPU."""
    N, K = w.shape
    v = w.cpu().float().view(N, K // 128, 128)
    n = -(-N // 128)
    top = torch.zeros((n * 128, K // 128))
    top[:N] = v.abs().amax(-1)
    top = top.view(n, 128, K // 128).amax(1)
    c, _ = quantise(v, top.repeat_interleave(128, 0)[:N])
    return c.view(torch.uint8).view(N, K), top / 448.0


def act_values(xq, sa):
    """What codes and scales of activations stand for, in 64 bits."""
    M, K = xq.shape
    return (xq.view(F8).double().view(M, K // 128, 128) * sa.double().t()[..., None]).view(M, K)


def weight_values(w8, sw):
    N, K = w8.shape
    return (w8.view(F8).double().view(N, K // 128, 128) * sw.double().repeat_interleave(128, 0)[:N, :, None]).view(N, K)


def product(x, w):
    """(x w^T in 64 bits, the bound of its fp32 form's error)."""
    return x @ w.t(), (140 + x.shape[1] // 128) * 2.0 ** -23 * (x.abs() @ w.abs().t())


def check_linear(y, x, w):
    ref, d = product(x, w)
    assert torch.all((y.double() - ref).abs() <= d + 2.0 ** -8 * (ref.abs() + d) + 1e-40)


def gated(x, wg, wu):
    """h = silu(g) u in 64 bits and the bound of its fp32 form's error.  |silu'| < 1.1; exp takes (2 + 1.5 |g|) 2^-23
    (2 ulp, and the product with log2 e rounded), sum, quotient and product three roundings more; below 2^-120 |u| the
    quotient may be 0."""
    g, dg = product(x, wg)
    u, du = product(x, wu)
    a = g * torch.sigmoid(g)
    d = 1.1 * dg * (u.abs() + du) + a.abs() * du + (8 + 2 * g.abs()) * 2.0 ** -23 * (a * u).abs() + 2.0 ** -118 * u.abs()
    return a * u, d


def check_codes(hq, sh, ref, d):
    """E4M3 codes with block scales of values that are off ref by d at most."""
    M, N = ref.shape
    top, dt = (t.view(M, N // 128, 128).amax(-1) for t in (ref.abs(), d))
    s = sh.double().t()
    assert torch.all((s - top / 448).abs() <= dt / 448 + 2.0 ** -22 * (top + dt) / 448 + 1e-45)
    s = s.repeat_interleave(128, 1)
    got = hq.view(F8).double() * s
    step = torch.maximum((ref.abs() + d) * 2.0 ** -4, s * 2.0 ** -10)
    assert torch.all((got - ref).abs() <= d + step * (1 + 2.0 ** -20) + 1e-44)


def check_bf16(h, ref, d):
    assert torch.all((h.double() - ref).abs() <= d + 2.0 ** -8 * (ref.abs() + d) + 1e-40)
