"""Rows into and out of the 4-bit KV cache: every bit against the definition."""
import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q, synthetic as syn
from gpuhelp import need_gpu, read_status, status
from layerref import pack, quantise_rows, values, words

pytestmark = pytest.mark.gpu


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def starts(lens, dev):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return ints(at, dev)


def rows_of(n, H, D, seed, dev):
    x = syn.activations(n * H, D, seed, device=dev, outlier_frac=0.02).view(n, H, D)
    return x.clone()


def expect(cache, k, v, lens, base):
    at = 0
    for b, (n, p) in enumerate(zip(lens, base)):
        for x, codes, sz in ((k, cache[0], cache[1]), (v, cache[2], cache[3])):
            c, s, z = quantise_rows(x[at:at + n])
            codes[b, :, p:p + n] = pack(c).transpose(0, 1)
            sz[b, :, p:p + n] = words(s, z).transpose(0, 1)
        at += n


def filled(B, H, T, D, dev):
    cache = q.kv4_cache(B, H, T, D, device=dev)
    for t in cache:
        t.fill_(0x5A)
    return cache


@pytest.mark.parametrize("H,D", [(1, 64), (8, 128), (3, 128), (4, 64)])
@pytest.mark.parametrize("lens,base,T", [([1], [0], 1), ([5, 5, 5], [7, 0, 11], 16), ([0, 33, 1, 0, 64], [9, 0, 99, 100, 36], 100),
                                         ([300], [17], 400)])
def test_append_and_load_bit_exact(H, D, lens, base, T):
    dev = need_gpu()
    B, n = len(lens), sum(lens)
    k, v = rows_of(n, H, D, 1, dev), rows_of(n, H, D, 2, dev)
    cache, want = filled(B, H, T, D, dev), filled(B, H, T, D, dev)
    st = status(dev)
    q.kv4_append(cache, k, v, starts(lens, dev), ints(base, dev), dev_status=st)
    assert read_status(st) == 0
    expect(want, k, v, lens, base)
    for got, ref in zip(cache, want):
        assert torch.equal(got, ref)
    ko, vo = q.kv4_load(cache, starts(lens, dev), ints(base, dev), n, dev_status=st)
    assert read_status(st) == 0
    at = 0
    for b, (m, p) in enumerate(zip(lens, base)):
        for o, codes, sz in ((ko, cache[0], cache[1]), (vo, cache[2], cache[3])):
            ref = values(codes[b, :, p:p + m], sz[b, :, p:p + m]).transpose(0, 1).to(torch.bfloat16)
            assert torch.equal(o[at:at + m], ref)
        at += m


def test_crafted_rows():
    """Ties to even, one sign only, a zero row, subnormal scales, the largest finite scale."""
    dev = need_gpu()
    D = 64
    x = torch.zeros((8, 1, D), device=dev)
    x[0, 0, :16] = torch.arange(16, device=dev).float()          # s = 1, z = 0
    x[0, 0, 16:22] = torch.tensor([0.5, 1.5, 2.5, 3.5, 13.5, 14.5], device=dev)
    x[1, 0] = -x[0, 0]                                           # z = 15
    x[2, 0, :3] = torch.tensor([-7.5, 7.5, 0.5], device=dev)     # -lo / s a tie
    x[4, 0, :2] = torch.tensor([1e-6, -3e-7], device=dev)        # scale an fp16 subnormal
    x[5, 0, :2] = torch.tensor([1e-9, 0.0], device=dev)          # scale 0 in fp16
    x[6, 0, :2] = torch.tensor([900000.0, -80000.0], device=dev)
    x[7, 0] = 3.0                                                # one value, away from 0
    x = x.to(torch.bfloat16)
    cache = filled(1, 1, 8, D, dev)
    st = status(dev)
    q.kv4_append(cache, x, x.flip(0).contiguous(), starts([8], dev), ints([0], dev), dev_status=st)
    assert read_status(st) == 0
    want = filled(1, 1, 8, D, dev)
    expect(want, x, x.flip(0), [8], [0])
    for got, ref in zip(cache, want):
        assert torch.equal(got, ref)
    assert int(want[1][0, 0, 3]) == 0 and int(want[1][0, 0, 5]) == 0 and 0 < int(want[1][0, 0, 4]) & 0xFFFF < 1024


def test_every_bf16_value_against_many_scales():
    """All finite bf16 magnitudes below the row's top, for rows of many tops: the division-free quotient."""
    dev = need_gpu()
    D, H = 128, 8
    g = torch.Generator(device=dev).manual_seed(3)
    bits = torch.randint(0x3000, 0x4300, (4096, H, D), generator=g, device=dev, dtype=torch.int32)
    sign = torch.randint(0, 2, bits.shape, generator=g, device=dev, dtype=torch.int32) << 15
    x = (bits | sign).to(torch.int16).view(torch.bfloat16)
    k = x.clone()
    k[:, :, 0] = k.abs().float().amax(-1).to(torch.bfloat16)
    cache, want = filled(1, H, 4096, D, dev), filled(1, H, 4096, D, dev)
    q.kv4_append(cache, k, x, starts([4096], dev), ints([0], dev))
    expect(want, k, x, [4096], [0])
    for got, ref in zip(cache, want):
        assert torch.equal(got, ref)


def test_rows_as_columns_of_a_fused_projection():
    dev = need_gpu()
    H, D, n, T = 4, 128, 11, 32
    y = syn.activations(n, (8 + 2 * H) * D, 7, device=dev)
    k, v = y[:, 8 * D:(8 + H) * D].view(n, H, D), y[:, (8 + H) * D:].view(n, H, D)
    a, b = filled(2, H, T, D, dev), filled(2, H, T, D, dev)
    q.kv4_append(a, k, v, starts([5, 6], dev), ints([3, 20], dev))
    q.kv4_append(b, k.contiguous(), v.contiguous(), starts([5, 6], dev), ints([3, 20], dev))
    for s, t in zip(a, b):
        assert torch.equal(s, t)


@pytest.mark.parametrize("start,base", [([0, 4, 8], [-1, 0]), ([0, 4, 8], [0, 13]), ([0, 4, 9], [0, 0]), ([-1, 4, 8], [0, 0]),
                                        ([0, 5, 3], [0, 0]), ([0, 4, 2 ** 31 - 1], [0, 2 ** 31 - 1])])
def test_ranges_that_do_not_hold(start, base):
    """Flagged; the sequence that is wrong stays untouched, on the way in and out."""
    dev = need_gpu()
    H, D, T = 2, 128, 16
    k, v = rows_of(8, H, D, 1, dev), rows_of(8, H, D, 2, dev)
    cache = filled(2, H, T, D, dev)
    st = status(dev)
    q.kv4_append(cache, k, v, ints(start, dev), ints(base, dev), dev_status=st)
    assert read_status(st) == q.ERR_RANGE
    for b in range(2):
        s0, s1, p = start[b], start[b + 1], base[b]
        if not (0 <= s0 <= s1 <= 8 and p >= 0 and p + s1 - s0 <= T):
            assert torch.all(cache[0][b] == 0x5A) and torch.all(cache[3][b] == 0x5A)
    st = status(dev)
    q.kv4_load(cache, ints(start, dev), ints(base, dev), 8, dev_status=st)
    assert read_status(st) == q.ERR_RANGE


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf"), 3e38])
def test_non_finite_rows_are_flagged(value):
    dev = need_gpu()
    k, v = rows_of(4, 2, 64, 1, dev), rows_of(4, 2, 64, 2, dev)
    v[2, 1, 33] = value
    cache = filled(1, 2, 8, 64, dev)
    st = status(dev)
    q.kv4_append(cache, k, v, starts([4], dev), ints([0], dev), dev_status=st)
    assert read_status(st) == q.ERR_NONFINITE
    want = filled(1, 2, 8, 64, dev)
    v[2, 1] = 0
    expect(want, k, v, [4], [0])
    assert torch.equal(cache[0], want[0]) and torch.equal(cache[2][:, 0], want[2][:, 0])


def test_no_rows():
    dev = need_gpu()
    cache = filled(2, 2, 4, 64, dev)
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=dev)
    q.kv4_append(cache, e, e, ints([0, 0, 0], dev), ints([0, 4], dev))
    k, v = q.kv4_load(cache, ints([0, 0, 0], dev), ints([0, 4], dev), 0)
    assert k.shape == (0, 2, 64) and torch.all(cache[0] == 0x5A)


@pytest.mark.parametrize("B", [1023, 1024, 1025, 2500])
def test_many_sequences_some_without_rows(B):
    """Around the number of sequences that the kernels look up in shared memory; runs of empty ones."""
    dev = need_gpu()
    H, D, T = 2, 64, 8
    lens = [0 if b % 7 in (1, 2, 3) else 1 + b % 5 for b in range(B)]
    base = [b % 3 for b in range(B)]
    n = sum(lens)
    k, v = rows_of(n, H, D, 1, dev), rows_of(n, H, D, 2, dev)
    cache, want = filled(B, H, T, D, dev), filled(B, H, T, D, dev)
    st = status(dev)
    q.kv4_append(cache, k, v, starts(lens, dev), ints(base, dev), dev_status=st)
    assert read_status(st) == 0
    expect(want, k, v, lens, base)
    for got, ref in zip(cache, want):
        assert torch.equal(got, ref)
    ko, vo = q.kv4_load(cache, starts(lens, dev), ints(base, dev), n, dev_status=st)
    assert read_status(st) == 0
    b = torch.tensor([i for i, m in enumerate(lens) for _ in range(m)], device=dev)
    p = torch.tensor([base[i] + j for i, m in enumerate(lens) for j in range(m)], device=dev)
    for o, codes, sz in ((ko, cache[0], cache[1]), (vo, cache[2], cache[3])):
        assert torch.equal(o, values(codes[b, :, p], sz[b, :, p]).to(torch.bfloat16))


def test_rows_before_and_after_the_sequences():
    """Rows of no sequence are left out on the way in and untouched on the way out."""
    dev = need_gpu()
    H, D, T = 3, 128, 32
    k, v = rows_of(40, H, D, 1, dev), rows_of(40, H, D, 2, dev)
    start, base = [3, 10, 30], [4, 1]
    cache, want = filled(2, H, T, D, dev), filled(2, H, T, D, dev)
    st = status(dev)
    q.kv4_append(cache, k, v, ints(start, dev), ints(base, dev), dev_status=st)
    assert read_status(st) == 0
    expect(want, k[3:30], v[3:30], [7, 20], base)
    for got, ref in zip(cache, want):
        assert torch.equal(got, ref)
    ko, vo = torch.full_like(k, 7.0), torch.full_like(v, 7.0)
    rc = q.qspec_kv4_load(*cache, ints(start, dev), ints(base, dev), 40, 2, H, T, D, ko, H * D, vo, H * D, st)
    assert rc == 0 and read_status(st) == 0
    for o in (ko, vo):
        assert torch.all(o[:3] == 7.0) and torch.all(o[30:] == 7.0) and not torch.any(torch.all((o[3:30] == 7.0).flatten(1), -1))
