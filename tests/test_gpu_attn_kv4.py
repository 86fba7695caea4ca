"""Attention over the 4-bit cache (qspec_attn_kv4) against the formula in 64 bits.

Tolerance of an output o = sum p v, with A = sum p |v|: the weights p s are
rounded to bf16 (half a step, 2^-8), the exponential is within 2^-12, a score
within d = 16 x 2^-24 x scale max_t s_t 143 sum |q| (fp32 sums of products with
codes held as 128 + c, or as smaller numbers), which counts twice (weight and sum): together
(2^-8 + 2^-12 + 2 d) A; and the output is rounded to bf16: 2^-8 |o|."""
import math

import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q, synthetic as syn
from gpuhelp import need_gpu, read_status, status
from layerref import attention, random_cache, values, words

pytestmark = pytest.mark.gpu


def queries(rows, Hq, D, seed, dev):
    return syn.activations(rows * Hq, D, seed, device=dev, outlier_frac=0.02).view(rows, Hq, D)


def check(qv, cache, lens, R, scale, o):
    B, H, T, D = cache[0].shape[0], cache[0].shape[1], cache[0].shape[2], qv.shape[2]
    G = qv.shape[1] // H
    for b, n in enumerate(lens):
        for h in range(H):
            k = values(cache[0][b, h, :n], cache[1][b, h, :n])
            v = values(cache[2][b, h, :n], cache[3][b, h, :n])
            s = (cache[1][b, h, :n] & 0xFFFF).to(torch.int16).view(torch.float16).double()
            for j in range(h * G, h * G + G):
                x = qv[b * R:b * R + R, j].double()
                ref, A = attention(x, k, v, n - R, scale)
                d = 16 * 2.0 ** -24 * abs(scale) * (float(s.max()) if n else 0.0) * 143 * x.abs().sum(-1, keepdim=True)
                tol = (2.0 ** -8 + 2.0 ** -12 + 2 * d) * A + 2.0 ** -8 * ref.abs() + 1e-30
                err = (o[b * R:b * R + R, j].double() - ref).abs()
                assert torch.all(err <= tol), (b, j, float((err - tol).max()), float((err / tol).max()))


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


@pytest.mark.parametrize("R", [1, 2, 5, 9, 17])
@pytest.mark.parametrize("H,G", [(1, 1), (2, 4), (4, 7), (1, 8), (3, 2)])
@pytest.mark.parametrize("D", [64, 128])
def test_rows_heads_and_lengths(R, H, G, D):
    dev = need_gpu()
    lens = [0, 1, 3, 15, 16, 17, 63, 64, 65, 128, 200, 257]
    T = 257
    cache = random_cache(len(lens), H, T, D, R + H, dev)
    x = queries(len(lens) * R, H * G, D, 11, dev)
    st = status(dev)
    o = q.attn_kv4(x, cache, ints(lens, dev), 1 / math.sqrt(D), dev_status=st)
    assert read_status(st) == 0
    check(x, cache, lens, R, 1 / math.sqrt(D), o)
    assert torch.all(o[:R] == 0)                                     # an empty cache


@pytest.mark.parametrize("B,R,H,G,D,T,lens", [(1, 1, 8, 4, 128, 20000, [19999]), (2, 5, 8, 4, 128, 5000, [4999, 1]),
                                              (3, 9, 4, 7, 128, 3001, [3001, 0, 2500]), (1, 17, 2, 8, 64, 9000, [8999]),
                                              (1, 1, 1, 1, 64, 40000, [40000]), (40, 1, 2, 4, 128, 700, None)])
def test_long_and_many(B, R, H, G, D, T, lens):
    dev = need_gpu()
    lens = lens or [(37 * b) % (T + 1) for b in range(B)]
    cache = random_cache(B, H, T, D, 5, dev)
    x = queries(B * R, H * G, D, 6, dev)
    st = status(dev)
    o = q.attn_kv4(x, cache, ints(lens, dev), 0.09, dev_status=st)
    assert read_status(st) == 0
    check(x, cache, lens, R, 0.09, o)


@pytest.mark.parametrize("scale", [0.0, 3.0, -0.5])
def test_scales(scale):
    """A flat softmax, a sharp one (scores of some hundreds), a negative scale."""
    dev = need_gpu()
    cache = random_cache(2, 2, 600, 128, 9, dev)
    x = queries(10, 8, 128, 10, dev)
    o = q.attn_kv4(x, cache, ints([600, 411], dev), scale)
    check(x, cache, [600, 411], 5, scale, o)


def test_places_past_the_length_do_not_matter():
    """Scale words of NaN and inf past the lengths, and past what each row sees."""
    dev = need_gpu()
    B, R, H, G, D, T, lens = 3, 5, 2, 4, 128, 300, [70, 2, 299]
    cache = random_cache(B, H, T, D, 1, dev)
    x = queries(B * R, H * G, D, 2, dev)
    ref = q.attn_kv4(x, cache, ints(lens, dev), 0.1)
    for b, n in enumerate(lens):
        for sz in (cache[1], cache[3]):
            sz[b, :, n:] = 0x7C007E00 if b else 0x7E007C00
        cache[0][b, :, n:] = 0xFF
    st = status(dev)
    o = q.attn_kv4(x, cache, ints(lens, dev), 0.1, dev_status=st)
    assert read_status(st) == 0 and torch.equal(o, ref)
    # a verify row's own future: only the rows that see position n - 1 change
    for b, n in enumerate(lens):
        if n:
            cache[3][b, :, n - 1] = 0x00007C00
    o2 = q.attn_kv4(x, cache, ints(lens, dev), 0.1).view(B, R, H * G, D)
    assert torch.equal(o2[:, :R - 1], o.view(B, R, H * G, D)[:, :R - 1])


def test_strided_queries_and_outputs():
    dev = need_gpu()
    B, R, H, G, D, T = 3, 3, 2, 4, 64, 90
    cache = random_cache(B, H, T, D, 1, dev)
    y = syn.activations(B * R, (H * G + 2 * H) * D, 2, device=dev)
    x = y[:, :H * G * D].view(B * R, H * G, D)
    buf = torch.full((B * R, H * G * D + 16), 5.0, dtype=torch.bfloat16, device=dev)
    out = buf[:, :H * G * D].view(B * R, H * G, D)
    n = ints([90, 33, 7], dev)
    o = q.attn_kv4(x, cache, n, 0.125, out=out)
    assert o is out and torch.all(buf[:, H * G * D:] == 5.0)
    assert torch.equal(out, q.attn_kv4(x.contiguous(), cache, n, 0.125))
    check(x, cache, [90, 33, 7], R, 0.125, out)


def test_one_workspace_for_many_calls_and_the_same_bits():
    """Any order of shapes on one workspace; the same call gives the same bits."""
    dev = need_gpu()
    ws = q.attn_kv4_workspace(16, 17, 32, 4, 128, dev)
    shapes = [(1, 1, 8, 4, 128, 6000), (16, 5, 4, 8, 128, 333), (2, 17, 4, 8, 64, 2000), (1, 1, 1, 1, 64, 3)]
    first = []
    for turn in range(3):
        for i, (B, R, H, G, D, T) in enumerate(shapes):
            assert q.qspec_attn_kv4_workspace_bytes(B, R, H * G, H, D) <= ws.numel()
            cache = random_cache(B, H, T, D, i, dev)
            x = queries(B * R, H * G, D, i, dev)
            lens = [T - (b * 31) % T for b in range(B)]
            o = q.attn_kv4(x, cache, ints(lens, dev), 0.1, workspace=ws)
            if turn == 0:
                check(x, cache, lens, R, 0.1, o)
                first.append(o)
            assert torch.equal(o, first[i])


def test_lengths_out_of_range():
    dev = need_gpu()
    cache = random_cache(3, 2, 50, 64, 1, dev)
    x = queries(6, 4, 64, 2, dev)
    out = torch.full((6, 4, 64), 9.0, dtype=torch.bfloat16, device=dev)
    st = status(dev)
    ws = q.attn_kv4_workspace(3, 2, 4, 2, 64, dev)
    q.attn_kv4(x, cache, ints([51, 50, -1], dev), 0.1, out=out, dev_status=st, workspace=ws)
    assert read_status(st) == q.ERR_RANGE
    assert torch.all(out[:2] == 9.0) and torch.all(out[4:] == 9.0)
    st = status(dev)
    o = q.attn_kv4(x, cache, ints([50, 50, 0], dev), 0.1, dev_status=st, workspace=ws)
    assert read_status(st) == 0 and torch.equal(o[2:4], out[2:4])
    check(x, cache, [50, 50, 0], 2, 0.1, o)


def test_cache_offsets_past_32_bits():
    """Codes of the last sequence start past 2^32 bytes."""
    dev = need_gpu()
    B, H, T, D, n = 17, 8, 524288, 128, 300
    cache = (torch.empty((B, H, T, D // 2), dtype=torch.uint8, device=dev), torch.empty((B, H, T), dtype=torch.int32, device=dev),
             torch.empty((B, H, T, D // 2), dtype=torch.uint8, device=dev), torch.empty((B, H, T), dtype=torch.int32, device=dev))
    small = random_cache(1, H, n, D, 1, dev)
    for big, t in zip(cache, small):
        big[-1, :, :n] = t[0]
    x = queries(B, H * 4, D, 2, dev)
    lens = [0] * (B - 1) + [n]
    st = status(dev)
    o = q.attn_kv4(x, cache, ints(lens, dev), 0.1, dev_status=st)
    assert read_status(st) == 0 and torch.all(o[:-1] == 0)
    check(x[-1:], small, [n], 1, 0.1, o[-1:])
    k = torch.zeros((2, H, D), dtype=torch.bfloat16, device=dev) + 1.5
    q.kv4_append(cache, k, k, ints([0] * B + [2], dev), ints([0] * (B - 1) + [T - 2], dev))
    back, _ = q.kv4_load(cache, ints([0] * B + [2], dev), ints([0] * (B - 1) + [T - 2], dev), 2)
    assert torch.equal(back, k)


def test_another_stream_and_a_graph():
    dev = need_gpu()
    B, R, H, G, D, T = 2, 5, 2, 4, 128, 1000
    cache = random_cache(B, H, T, D, 1, dev)
    x = queries(B * R, H * G, D, 2, dev)
    n = ints([1000, 700], dev)
    ref = q.attn_kv4(x, cache, n, 0.1)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o = q.attn_kv4(x, cache, n, 0.1)
    s.synchronize()
    assert torch.equal(o, ref)
    ws, out = q.attn_kv4_workspace(B, R, H * G, H, D, dev), torch.zeros_like(x)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for _ in range(3):
            q.attn_kv4(x, cache, n, 0.1, workspace=ws, out=out)
    for lens in ([1000, 700], [5, 999], [0, 64]):
        n.copy_(ints(lens, dev))
        g.replay()
        torch.cuda.synchronize()
        check(x, cache, lens, R, 0.1, out)


@pytest.mark.parametrize("B,R,H,G,D,T", [(16, 1, 8, 4, 128, 4096), (16, 5, 8, 4, 128, 4090), (8, 9, 4, 7, 128, 4001),
                                         (6, 17, 2, 8, 64, 5000), (70, 2, 3, 4, 64, 900), (100, 9, 1, 2, 128, 1300)])
def test_several_tiles_of_a_group_and_several_tasks_of_a_share(B, R, H, G, D, T):
    """Each width of the products with every stage used many times over, and shares that end and begin inside tasks."""
    dev = need_gpu()
    lens = [T - (b * 997) % (T - T // 8) for b in range(B)]
    cache = random_cache(B, H, T, D, 21, dev)
    x = queries(B * R, H * G, D, 22, dev)
    st = status(dev)
    o = q.attn_kv4(x, cache, ints(lens, dev), 1 / math.sqrt(D), dev_status=st)
    assert read_status(st) == 0
    check(x, cache, lens, R, 1 / math.sqrt(D), o)


@pytest.mark.parametrize("R,G", [(1, 1), (5, 4), (9, 7)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("at", [1, 130, 777])
def test_a_score_far_above_the_first_position(R, G, D, at):
    """The first position's score is far below a later one's: the segment is taken again."""
    dev = need_gpu()
    T = 800
    cache = random_cache(1, 1, T, D, 31, dev, s_lo=0.01, s_hi=0.02)
    # values 15 s = 3 at position `at`, -3 at the first, rows of ones: scores of 3 D and -3 D times the scale
    cache[0][0, 0, at], cache[1][0, 0, at] = 0xFF, words(torch.tensor(0.2, device=dev), torch.tensor(0.0, device=dev))
    cache[0][0, 0, 0], cache[1][0, 0, 0] = 0x00, words(torch.tensor(0.2, device=dev), torch.tensor(15.0, device=dev))
    x = (queries(R, G, D, 32, dev).float() * 0.05 + 1.0).to(torch.bfloat16)
    scale = 100.0 / (3 * D)
    st = status(dev)
    o = q.attn_kv4(x, cache, ints([T], dev), scale, dev_status=st)
    assert read_status(st) == 0
    check(x, cache, [T], R, scale, o)


@pytest.mark.parametrize("B,R,H,G,D,n", [(1, 1, 8, 4, 128, 8100), (1, 5, 8, 4, 128, 1000), (16, 5, 8, 4, 128, 1000), (19, 1, 8, 4, 128, 515),
                                         (8, 9, 4, 7, 128, 2000), (2, 3, 1, 2, 64, 513), (38, 17, 4, 8, 64, 700)])
def test_sequences_of_one_length(B, R, H, G, D, n):
    """Tasks in equal parts, whole tasks to a CTA, and the first size past that; an invalid sequence among them."""
    dev = need_gpu()
    lens = [n - b % 3 for b in range(B)]
    cache = random_cache(B, H, n, D, 41, dev)
    x = queries(B * R, H * G, D, 42, dev)
    st = status(dev)
    o = q.attn_kv4(x, cache, ints(lens, dev), 1 / math.sqrt(D), dev_status=st)
    assert read_status(st) == 0
    check(x, cache, lens, R, 1 / math.sqrt(D), o)
    if B > 1:
        lens[B // 2] = -1
        o2 = q.attn_kv4(x, cache, ints(lens, dev), 1 / math.sqrt(D), out=torch.full_like(o, 9.0), dev_status=st)
        assert read_status(st) == q.ERR_RANGE
        lens[B // 2] = 0
        assert torch.all(o2.view(B, R, -1)[B // 2] == 9.0)
        o2.view(B, R, -1)[B // 2] = 0
        check(x, cache, lens, R, 1 / math.sqrt(D), o2)
