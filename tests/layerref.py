"""Plain 64-bit forms of the 4-bit cache and of attention, for the tests."""
import torch


def quantise_rows(x):
    """[..., D] bf16 -> (codes int64, s fp64 (an fp16 value), z fp64): s = fp16((hi - lo) / 15) through fp32, the
    quotients as IEEE fp32 ones, ties to even."""
    f = x.float()
    lo, hi = f.amin(-1).clamp(max=0.0), f.amax(-1).clamp(min=0.0)
    s = ((hi - lo) / 15.0).to(torch.float16).float()
    one = torch.where(s > 0, s, torch.ones_like(s))
    z = torch.where(s > 0, torch.round(-lo / one).clamp(0, 15), torch.zeros_like(s))
    c = (torch.round(f / one[..., None]) + z[..., None]).clamp(0, 15)
    c = torch.where(s[..., None] > 0, c, torch.zeros_like(c))
    return c.to(torch.int64), s.double(), z.double()


def pack(codes):
    c = codes.to(torch.uint8)
    return c[..., 0::2] | (c[..., 1::2] << 4)


def words(s, z):
    lo = s.to(torch.float16).view(torch.int16).to(torch.int32) & 0xFFFF
    return lo | (z.to(torch.float16).view(torch.int16).to(torch.int32) << 16)


def values(codes, word):
    """Packed bytes [..., D/2] and words [...] -> fp64 values [..., D]."""
    s = (word & 0xFFFF).to(torch.int16).view(torch.float16).double()
    z = ((word >> 16) & 0xFFFF).to(torch.int16).view(torch.float16).double()
    c = torch.stack((codes & 15, codes >> 4), dim=-1).flatten(-2).double()
    return s[..., None] * (c - z[..., None])


def random_cache(B, H, T, D, seed, dev, s_lo=0.05, s_hi=0.3):
    g = torch.Generator(device=dev).manual_seed(seed)
    out = []
    for _ in range(2):
        codes = torch.randint(0, 256, (B, H, T, D // 2), generator=g, device=dev, dtype=torch.uint8)
        s = torch.rand((B, H, T), generator=g, device=dev) * (s_hi - s_lo) + s_lo
        z = torch.randint(0, 16, (B, H, T), generator=g, device=dev)
        out += [codes, words(s, z)]
    return tuple(out)


def attention(q, k, v, first, scale):
    """One head: q [n, D], k, v [m, D] in fp64; row i sees keys 0 .. first + i.  Returns (o, A): A = sum p |v|,
    what an error of the weights is measured by.  Rows that see nothing are 0."""
    n, m = q.shape[0], k.shape[0]
    seen = torch.arange(m, device=q.device)[None, :] <= torch.arange(n, device=q.device)[:, None] + first
    a = torch.where(seen, (q @ k.T) * scale, torch.full((), -torch.inf, dtype=torch.float64, device=q.device))
    top = a.amax(-1, keepdim=True) if m else torch.zeros((n, 1), dtype=torch.float64, device=q.device)
    e = torch.exp(a - torch.where(torch.isfinite(top), top, torch.zeros_like(top)))
    t = e.sum(-1, keepdim=True)
    p = e / torch.where(t > 0, t, torch.ones_like(t))
    vz = torch.where(torch.isfinite(v), v, torch.zeros_like(v))
    return p @ vz, p @ vz.abs()
