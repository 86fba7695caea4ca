"""E4M3 with a scale for each block of 128: quantisers (every bit), the linear and the gated product (against 64 bits,
the bounds of blockref.py)."""
import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q, synthetic as syn
from blockref import (act_codes, act_values, check_bf16, check_codes, check_linear, gated, weight_codes, weight_values)
from gpuhelp import need_gpu, read_status, status

pytestmark = pytest.mark.gpu


def acts(M, K, seed, dev, std=1.0):
    """Rows of different sizes with outlier channels; some blocks of zeros."""
    x = syn.activations(M, K, seed, device=dev, outlier_frac=0.01).float()
    x *= (0.25 + torch.arange(M, device=dev)[:, None] % 5) * std
    if M > 2:
        x[1, :128] = 0.0
    return x.to(torch.bfloat16)


def parent(N, K, seed, dev, std=0.03):
    w = syn.activations(N, K, seed, device=dev).float() * std
    if N > 3:
        w[: min(N, 128), K - 128:] = 0.0               # a block of zeros
        w[N // 2] *= 16.0
    return w.to(torch.float16)


def same(a, b):
    return torch.equal(a.cpu().view(torch.uint8), b.cpu().view(torch.uint8))


@pytest.mark.parametrize("M,K", [(1, 128), (2, 384), (5, 4096), (33, 640), (40, 1152), (257, 14336), (3000, 1408)])
def test_activation_codes(M, K):
    dev = need_gpu()
    x, st = acts(M, K, M + K, dev), status(dev)
    xq, sa = q.quant_act_fp8_block(x, dev_status=st)
    assert read_status(st) == 0
    want = act_codes(x)
    assert same(xq, want[0]) and same(sa, want[1])


@pytest.mark.parametrize("N,K", [(1, 128), (127, 256), (128, 640), (129, 1152), (300, 4096), (1000, 384)])
def test_weight_codes(N, K):
    dev = need_gpu()
    w, st = parent(N, K, N + K, dev), status(dev)
    w8, sw = q.quant_weights_fp8_block(w, dev_status=st)
    assert read_status(st) == 0
    want = weight_codes(w)
    assert same(w8, want[0]) and same(sw, want[1])


@pytest.mark.parametrize("scale", [2.0 ** 120, 2.0 ** 79, 2.0 ** 70, 2.0 ** -60, 2.0 ** -73, 2.0 ** -90, 2.0 ** -126, 2.0 ** -133])
def test_activation_codes_of_extreme_magnitudes(scale):
    """Scales on both sides of where the quotient takes the division, subnormal ones among them."""
    dev = need_gpu()
    x = (acts(9, 512, 3, dev).float() * scale).to(torch.bfloat16)
    st = status(dev)
    xq, sa = q.quant_act_fp8_block(x, dev_status=st)
    assert read_status(st) == 0
    want = act_codes(x)
    assert same(sa, want[1]) and same(xq, want[0])


def over_all_maxima(bits, top_bits, dtype, dev):
    """Blocks of 128 that pair every value of `bits` with every maximum of `top_bits` that is not below it."""
    v = torch.tensor(bits, dtype=torch.int32).to(torch.int16).view(dtype).to(dev)
    blocks = []
    for t in top_bits:
        top = torch.tensor([t], dtype=torch.int32).to(torch.int16).view(dtype).to(dev)
        x = v[v.abs() <= top]
        n = -(-len(x) // 127)
        pad = torch.zeros(n * 127, dtype=dtype, device=dev)
        pad[:len(x)] = x
        blocks.append(torch.cat([top.expand(n, 1), pad.view(n, 127)], dim=1))
    return torch.cat(blocks)


def test_every_bf16_value_over_every_scale():
    """All 128 significands of a maximum with all values of 26 binades below it, of either sign, zeros and subnormal codes among
    them: code and quotient are the division's."""
    dev = need_gpu()
    bits = [sign | (e << 7) | f for sign in (0, 0x8000) for e in range(102, 129) for f in range(128)] + [0, 0x8000, 1, 0x8001]
    x = over_all_maxima(bits, [(127 << 7) | f for f in range(128)] + [(128 << 7)], torch.bfloat16, dev)
    xq, sa = q.quant_act_fp8_block(x)
    v = x.float()
    s = v.abs().amax(-1) / torch.tensor(448.0, device=dev)      # (by a number it would be times 1 / 448)
    want = (v / s[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    assert torch.equal(sa[0], s) and torch.equal(xq, want.view(torch.uint8))


def test_every_fp16_value_over_every_scale():
    """All 1024 significands of a maximum with all values of 20 binades, as weights (a block's values in its 128 rows)."""
    dev = need_gpu()
    bits = [sign | (e << 10) | f for sign in (0, 0x8000) for e in range(0, 17) for f in range(0, 1024)]
    for part in range(0, 1024, 64):
        x = over_all_maxima(bits, [(15 << 10) | f for f in range(part, part + 64)], torch.float16, dev)
        n = x.shape[0]
        w = torch.zeros((128, n * 128), dtype=torch.float16, device=dev)
        w[5] = x.reshape(-1)
        w8, sw = q.quant_weights_fp8_block(w)
        v = x.float()
        s = v.abs().amax(-1) / torch.tensor(448.0, device=dev)      # (by a number it would be times 1 / 448)
        want = (v / s[:, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
        assert torch.equal(sw[0], s) and torch.equal(w8[5].view(n, 128), want.view(torch.uint8))
        assert int(w8.count_nonzero()) == int(w8[5].count_nonzero())


@pytest.mark.parametrize("off", [0, 8])
def test_addresses_on_16_bytes(off):
    """Rows that begin between multiples of 32 bytes take their own way."""
    dev = need_gpu()
    M, K = 37, 640
    wide = torch.zeros((M, K + 24), dtype=torch.bfloat16, device=dev)
    wide[:, off:off + K] = acts(M, K, 2, dev)
    x = wide[:, off:off + K]
    st = status(dev)
    xq, sa = q.quant_act_fp8_block(x, dev_status=st)
    want = act_codes(x)
    assert read_status(st) == 0 and same(xq, want[0]) and same(sa, want[1])
    flat = torch.zeros(M * K + 16, dtype=torch.float16, device=dev)
    flat[off:off + M * K] = parent(M, K, 3, dev).reshape(-1)
    w = flat[off:off + M * K].view(M, K)
    w8, sw = q.quant_weights_fp8_block(w, dev_status=st)
    want = weight_codes(w)
    assert read_status(st) == 0 and same(w8, want[0]) and same(sw, want[1])


def test_rows_and_scales_apart():
    """Rows and rows of scales further apart than they are long: what lies between stays as it was."""
    dev = need_gpu()
    M, K, ldx, lds = 37, 640, 704, 41
    wide = torch.full((M, ldx), float("nan"), dtype=torch.bfloat16, device=dev)
    wide[:, :K] = acts(M, K, 1, dev)
    xq = torch.empty((M, K), dtype=torch.uint8, device=dev)
    sa = torch.full((K // 128, lds), -7.0, device=dev)
    st = status(dev)
    assert q.qspec_quant_act_fp8_block(wide, M, K, ldx, xq, sa, lds, st) == 0 and read_status(st) == 0
    want = act_codes(wide[:, :K])
    assert same(xq, want[0]) and same(sa[:, :M].contiguous(), want[1]) and torch.all(sa[:, M:] == -7.0)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
def test_quantisers_flag_what_is_not_finite(value):
    dev = need_gpu()
    x = acts(20, 384, 5, dev)
    want = act_codes(x)
    x[7, 130] = value
    st = status(dev)
    xq, sa = q.quant_act_fp8_block(x, dev_status=st)
    assert read_status(st) == q.ERR_NONFINITE and not torch.isfinite(sa[1, 7])
    sa[1, 7] = want[1][1, 7]
    assert same(sa, want[1]) and same(xq[8:], want[0][8:])            # the other blocks are what they were
    w = parent(200, 256, 6, dev)
    want = weight_codes(w)
    w[150, 3] = value
    st = status(dev)
    w8, sw = q.quant_weights_fp8_block(w, dev_status=st)
    assert read_status(st) == q.ERR_NONFINITE and not torch.isfinite(sw[1, 0])
    assert same(w8[:128], want[0][:128]) and same(w8[:, 128:].contiguous(), want[0][:, 128:].contiguous())


def codes(M, K, seed, dev):
    return q.quant_act_fp8_block(acts(M, K, seed, dev))


SHAPES = [(1, 128, 128), (1, 1, 128), (2, 300, 384), (1, 4096, 1152), (5, 1000, 4096), (15, 129, 14336), (16, 128, 256),
          (17, 127, 640), (31, 640, 1408), (33, 257, 2048), (64, 384, 896), (65, 100, 1152), (80, 1024, 4096), (127, 130, 256),
          (128, 512, 640), (129, 384, 512), (255, 256, 128), (257, 300, 1024), (288, 1152, 1408), (600, 640, 768), (1025, 257, 384), (2500, 2560, 256)]


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_linear(M, N, K):
    dev = need_gpu()
    xq, sa = codes(M, K, M, dev)
    w8, sw = q.quant_weights_fp8_block(parent(N, K, N, dev))
    st = status(dev)
    y = q.linear_fp8_block(xq, sa, w8, sw, dev_status=st)
    assert read_status(st) == 0
    check_linear(y, act_values(xq, sa), weight_values(w8, sw))


@pytest.mark.parametrize("M,N,K", [(M, -(-N // 128) * 128, K) for M, N, K in SHAPES])
def test_gated(M, N, K):
    dev = need_gpu()
    xq, sa = codes(M, K, M + 1, dev)
    wg, wu = (q.quant_weights_fp8_block(parent(N, K, N + i, dev)) for i in (1, 2))
    st = status(dev)
    hq, sh, h = q.gated_fp8_block(xq, sa, *wg, *wu, want_bf16=True, dev_status=st)
    assert read_status(st) == 0
    ref, d = gated(act_values(xq, sa), weight_values(*wg), weight_values(*wu))
    check_codes(hq, sh, ref, d)
    check_bf16(h, ref, d)
    # one output without the other: the same bits
    a, b = q.gated_fp8_block(xq, sa, *wg, *wu), q.gated_fp8_block(xq, sa, *wg, *wu, want_fp8=False, want_bf16=True)
    assert torch.equal(a[0], hq) and torch.equal(a[1], sh) and a[2] is None
    assert torch.equal(b[2], h) and b[0] is None and b[1] is None


@pytest.mark.parametrize("M,std", [(5, 30.0), (40, 3000.0), (300, 30.0), (300, 3000.0)])
def test_gated_far_from_zero(M, std):
    """Gates where exp passes fp32 on one side and vanishes on the other."""
    dev = need_gpu()
    N, K = 256, 512
    xq, sa = q.quant_act_fp8_block(acts(M, K, 8, dev, std=std))
    wg, wu = (q.quant_weights_fp8_block(parent(N, K, i, dev)) for i in (1, 2))
    st = status(dev)
    hq, sh, h = q.gated_fp8_block(xq, sa, *wg, *wu, want_bf16=True, dev_status=st)
    assert read_status(st) == 0
    ref, d = gated(act_values(xq, sa), weight_values(*wg), weight_values(*wu))
    check_codes(hq, sh, ref, d)
    check_bf16(h, ref, d)


@pytest.mark.parametrize("M", [3, 70, 300])
def test_blocks_of_zeros(M):
    """Scales of 0 in every row of weights and tokens: outputs, codes and scales of 0."""
    dev = need_gpu()
    N, K = 256, 384
    xq, sa = q.quant_act_fp8_block(torch.zeros((M, K), dtype=torch.bfloat16, device=dev))
    wg, wu = (q.quant_weights_fp8_block(parent(N, K, i, dev)) for i in (1, 2))
    for a, b in ((xq, sa), codes(M, K, 9, dev)):
        z = q.quant_weights_fp8_block(torch.zeros((N, K), dtype=torch.float16, device=dev)) if a is not xq else wg
        assert torch.all(q.linear_fp8_block(a, b, *z) == 0)
        hq, sh, h = q.gated_fp8_block(a, b, *z, *wu, want_bf16=True)
        assert not hq.any() and not sh.any() and torch.all(h == 0)


@pytest.mark.parametrize("M", [7, 64, 130, 513])
@pytest.mark.parametrize("ldy", [391, 392, 400])
def test_outputs_apart(M, ldy):
    """Leading dimensions wider than the rows, odd ones and such on 16 bytes among them, codes on 16 bytes, scales further
    apart than tokens: nothing else is written, and what stands past the last token is not read."""
    dev = need_gpu()
    N, K, lds, ldh = 384, 640, M + 3, M + 5
    xq, sa0 = codes(M, K, 4, dev)
    sa = torch.full((K // 128, lds), float("nan"), device=dev)
    sa[:, :M] = sa0
    wg, wu = (q.quant_weights_fp8_block(parent(N, K, i, dev)) for i in (1, 2))
    y = torch.full((M, ldy), 7.0, dtype=torch.bfloat16, device=dev)
    st = status(dev)
    assert q.qspec_linear_fp8_block(xq, sa, lds, *wg, M, N - 1, K, y, ldy, st) == 0 and read_status(st) == 0
    assert torch.all(y[:, N - 1:] == 7.0)
    check_linear(y[:, :N - 1], act_values(xq, sa0), weight_values(*wg)[:N - 1])
    flat = torch.full((16 + (M + 1) * N,), 9, dtype=torch.uint8, device=dev)
    hq = flat[16:].view(M + 1, N)
    sh = torch.full((N // 128, ldh), -7.0, device=dev)
    h = torch.full((M, ldy), 7.0, dtype=torch.bfloat16, device=dev)
    assert q.qspec_gated_fp8_block(xq, sa, lds, *wg, *wu, M, N, K, hq, sh, ldh, h, ldy, st) == 0 and read_status(st) == 0
    assert torch.all(hq[M] == 9) and torch.all(flat[:16] == 9) and torch.all(sh[:, M:] == -7.0) and torch.all(h[:, N:] == 7.0)
    ref, d = gated(act_values(xq, sa0), weight_values(*wg), weight_values(*wu))
    check_codes(hq[:M], sh[:, :M], ref, d)
    check_bf16(h[:, :N], ref, d)


@pytest.mark.parametrize("M", [2, 300])
def test_products_that_pass_fp32_are_flagged(M):
    dev = need_gpu()
    N, K = 128, 256
    x = torch.full((M, K), 2.0 ** 100, dtype=torch.bfloat16, device=dev)
    x[0] = 1.0
    xq, sa = q.quant_act_fp8_block(x)
    w = q.quant_weights_fp8_block(torch.full((N, K), 1.0, dtype=torch.float16, device=dev))
    st = status(dev)
    hq, sh, _ = q.gated_fp8_block(xq, sa, *w, *w, dev_status=st)
    assert read_status(st) == q.ERR_NONFINITE
    assert not torch.isfinite(sh[0, 1:]).any()
    ref, d = gated(act_values(xq[:1], sa[:, :1]), weight_values(*w), weight_values(*w))      # (the other rows are what they were)
    check_codes(hq[:1], sh[:, :1], ref, d)


@pytest.mark.parametrize("M,N,K", [(1, 4096, 14336), (5, 14336, 4096), (288, 3584, 18944), (100, 18944, 3584)])
def test_the_models_shapes_in_sampled_channels(M, N, K):
    dev = need_gpu()
    xq, sa = codes(M, K, 1, dev)
    g = torch.Generator(device=dev).manual_seed(2)
    w8, sw = q.quant_weights_fp8_block((torch.randn((N, K), generator=g, device=dev) * 0.02).to(torch.float16))
    y = q.linear_fp8_block(xq, sa, w8, sw)
    for n in (0, 128 * (N // 256), N - 128):
        check_linear(y[:, n:n + 128], act_values(xq, sa), weight_values(w8[n:n + 128], sw[n // 128:n // 128 + 1]))


@pytest.mark.parametrize("M", [513, 531, 546, 640])
@pytest.mark.parametrize("N", [3840, 2304, 1792, 768])
@pytest.mark.parametrize("K", [2048, 4096])
def test_parts_of_k_that_meet(M, N, K):
    """Tiles in two, three, four and more parts of K, the last tile of 1, 19, 34 and 128 tokens."""
    dev = need_gpu()
    xq, sa = codes(M, K, M + N, dev)
    w8, sw = q.quant_weights_fp8_block(parent(N, K, N, dev))
    st = status(dev)
    y = torch.full((M + 3, N), -7.0, dtype=torch.bfloat16, device=dev)
    q.linear_fp8_block(xq, sa, w8, sw, out=y[:M], dev_status=st)
    assert read_status(st) == 0
    check_linear(y[:M], act_values(xq, sa), weight_values(w8, sw))
    assert torch.all(y[M:] == -7.0)                                   # rows behind the last are left as they were
    z = torch.full((M + 1, N + 1), -7.0, dtype=torch.bfloat16, device=dev)
    assert q.qspec_linear_fp8_block(xq, sa, M, w8, sw, M, N, K, z, N + 1, st) == 0 and read_status(st) == 0
    assert torch.equal(z[:M, :N], y[:M]) and torch.all(z[M:] == -7.0) and torch.all(z[:, N:] == -7.0)


# few tokens with K in three, five and six parts, one CTA and two to an SM; more channels than fit the machine at once; long K
PARTS = [(1, 10240, 1536), (7, 6144, 2560), (16, 5120, 2048), (64, 5120, 2048), (100, 5120, 1280), (90, 2560, 2560), (100, 20480, 256), (40, 39424, 128),
         (128, 14336, 4096), (30, 5120, 1280), (20, 19584, 256), (80, 2048, 4096), (33, 1024, 2048), (49, 9216, 512), (64, 4096, 1152), (51, 9856, 256),
         (1, 4736, 4096), (9, 9600, 2048)]


@pytest.mark.parametrize("M,N,K", PARTS)
@pytest.mark.parametrize("is_gated", [False, True])
def test_few_tokens_in_odd_parts_and_wide(M, N, K, is_gated):
    dev = need_gpu()
    xq, sa = codes(M, K, M + 1, dev)
    w, v = (q.quant_weights_fp8_block(parent(N, K, N + i, dev)) for i in (1, 2))
    st = status(dev)
    if is_gated:
        hq, sh, h = q.gated_fp8_block(xq, sa, *w, *v, want_bf16=True, dev_status=st)
        ref, d = gated(act_values(xq, sa), weight_values(*w), weight_values(*v))
        check_codes(hq, sh, ref, d)
        check_bf16(h, ref, d)
    else:
        check_linear(q.linear_fp8_block(xq, sa, *w, dev_status=st), act_values(xq, sa), weight_values(*w))
    assert read_status(st) == 0


@pytest.mark.parametrize("M,N,K", [(640, 1920, 5120), (520, 1152, 4096), (513, 896, 4096), (200, 512, 4096), (130, 14336, 4096), (300, 8192, 4096)])
def test_gated_parts_of_k_that_meet(M, N, K):
    """Tiles in two, three, four and eight parts of K, and tiles behind a full round in two and three."""
    dev = need_gpu()
    xq, sa = codes(M, K, M + N, dev)
    wg, wu = (q.quant_weights_fp8_block(parent(N, K, N + i, dev)) for i in (1, 2))
    st = status(dev)
    flat = torch.full((M + 1, N), 9, dtype=torch.uint8, device=dev)
    sh = torch.full((N // 128, M + 2), -7.0, device=dev)
    h = torch.full((M + 1, N + 1), -7.0, dtype=torch.bfloat16, device=dev)
    assert q.qspec_gated_fp8_block(xq, sa, M, *wg, *wu, M, N, K, flat, sh, M + 2, h, N + 1, st) == 0 and read_status(st) == 0
    ref, d = gated(act_values(xq, sa), weight_values(*wg), weight_values(*wu))
    check_codes(flat[:M], sh[:, :M], ref, d)
    check_bf16(h[:M, :N], ref, d)
    assert torch.all(flat[M] == 9) and torch.all(sh[:, M:] == -7.0) and torch.all(h[M] == -7.0) and torch.all(h[:, N:] == -7.0)
    again = q.gated_fp8_block(xq, sa, *wg, *wu, want_bf16=True)
    assert torch.equal(again[0], flat[:M]) and torch.equal(again[1], sh[:, :M]) and torch.equal(again[2], h[:M, :N])


def test_a_token_does_not_depend_on_the_others():
    """Gates far below zero, or not finite, in one token of a tile: the other tokens keep their bits."""
    dev = need_gpu()
    M, N, K = 300, 256, 512
    x = acts(M, K, 8, dev)
    wg, wu = (q.quant_weights_fp8_block(parent(N, K, i, dev)) for i in (1, 2))
    want = q.gated_fp8_block(*q.quant_act_fp8_block(x), *wg, *wu, want_bf16=True)
    x[17] *= 4000.0
    x[200, 3] = float("nan")
    got = q.gated_fp8_block(*q.quant_act_fp8_block(x), *wg, *wu, want_bf16=True)
    keep = [m for m in range(M) if m not in (17, 200)]
    assert torch.equal(got[0][keep], want[0][keep]) and torch.equal(got[1][:, keep], want[1][:, keep]) and torch.equal(got[2][keep], want[2][keep])
    assert torch.isnan(got[1][:, 200]).all()


def test_offsets_past_32_bits():
    """Tensors of more than 2^32 values: their last rows against the definitions."""
    dev = need_gpu()
    M, K = 263000, 16384
    x = torch.zeros((M, K), dtype=torch.bfloat16, device=dev)
    x[-5:] = acts(5, K, 1, dev)
    xq, sa = q.quant_act_fp8_block(x)
    want = act_codes(x[-5:])
    assert same(xq[-5:], want[0]) and same(sa[:, -5:].contiguous(), want[1])
    w = x.view(torch.int16).zero_().view(torch.float16)                       # (the same memory as weights)
    w[-200:] = parent(200, K, 2, dev)
    w8, sw = q.quant_weights_fp8_block(w)
    n0 = (M - 200) // 128 * 128
    want = weight_codes(w[n0:])
    assert same(w8[n0:], want[0]) and same(sw[n0 // 128:], want[1])
    del x, w, xq, sa
    a = codes(3, K, 3, dev)
    y = q.linear_fp8_block(*a, w8, sw)
    check_linear(y[:, n0:], act_values(*a), weight_values(w8[n0:], sw[n0 // 128:]))
    del w8, sw, y
    M, N, K = 66000, 66048, 128
    xq, sa = codes(M, K, 4, dev)
    wg, wu = (q.quant_weights_fp8_block(parent(N, K, i, dev)) for i in (5, 6))
    y = q.linear_fp8_block(xq, sa, *wg)
    xs, gs, us = act_values(xq[-200:], sa[:, -200:]), weight_values(wg[0][-256:], wg[1][-2:]), weight_values(wu[0][-256:], wu[1][-2:])
    check_linear(y[-200:, -256:], xs, gs)
    hq, sh, h = q.gated_fp8_block(xq, sa, *wg, *wu, want_bf16=True)
    ref, d = gated(xs, gs, us)
    check_codes(hq[-200:, -256:], sh[-2:, -200:], ref, d)
    check_bf16(h[-200:, -256:], ref, d)


FIRST = """
import sys; sys.path[:0] = [%r, %r]
import torch
from quantized_speculative_decoding_shared_gb300 import binding as q
dev = torch.device('cuda')
g = torch.Generator(device=dev).manual_seed(1)
make = lambda r, c: torch.randint(0, 100, (r, c), generator=g, device=dev, dtype=torch.uint8)
K, N = 512, 384
rows = (3, 40, 100, 300)
xs = [(make(m, K), torch.rand((K // 128, m), generator=g, device=dev)) for m in rows]
w = [(make(N, K), torch.rand((N // 128, K // 128), generator=g, device=dev)) for _ in range(2)]
def program():
    out = []
    for x in xs:
        out += [q.linear_fp8_block(*x, *w[0]), *q.gated_fp8_block(*x, *w[0], *w[1])[:2]]
    return out
torch.cuda.synchronize()
s, gr = torch.cuda.Stream(), torch.cuda.CUDAGraph()
with torch.cuda.graph(gr, stream=s):
    got = program()
gr.replay()
torch.cuda.synchronize()
want = program()
torch.cuda.synchronize()
print('same', all(torch.equal(a, b) for a, b in zip(got, want)))
"""


def test_the_first_calls_of_a_process_are_captured():
    import os
    import subprocess
    import sys
    need_gpu()
    here = os.path.dirname(os.path.abspath(__file__))
    r = subprocess.run([sys.executable, "-c", FIRST % (os.path.dirname(here), here)], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same True" in r.stdout, r.stdout + r.stderr
