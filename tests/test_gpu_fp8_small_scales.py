"""E4M3 codes beside scales that are subnormal or 0: a code is E4M3(value / the scale as stored), and 0 where that is 0.

Tolerances.  A stored scale is the fp32 quotient: the norm's bound (64 x 2^-24 of it, as in test_gpu_norm_block.py) and half
a subnormal step, 2^-150, for itself and for the maximum that it is the 448th of.  In the norm a product h w below 2^-126 is rounded to a multiple of 2^-149: 2^-150 / rms in y.  A code against value / stored scale, in 64 bits: half an E4M3 step (2^-4 of it, 2^-10 below 2^-6)
and the value's own bound; at most 448 by saturation, so that a scale that was rounded down may leave the largest values short."""
import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q, synthetic as syn
from blockref import F8, act_values, gated, weight_values
from gpuhelp import need_gpu, read_status, status

pytestmark = pytest.mark.gpu
EPS = 1e-5


def check(codes, scales, ref, d):
    """codes and ref [..., n], scales [...] stored, d the bound of the values behind the codes."""
    top = ref.abs().amax(-1)
    assert torch.all((scales - top / 448).abs() <= d.amax(-1) / 448 + 64 * 2.0 ** -24 * top / 448 + 2.0 ** -150 * (1 + 1 / 448))
    none = scales == 0
    assert not codes[none].view(torch.uint8).any()
    s = scales[~none][..., None]
    v, dv, c = ref[~none] / s, d[~none] / s, codes[~none].double()
    want = v.clamp(-448, 448)
    assert torch.all((c - want).abs() <= torch.clamp((v.abs() + dv) * 2.0 ** -4, min=2.0 ** -10) + dv + v.abs() * 2.0 ** -18)


def norm_ref(x, w, eps):
    """y in 64 bits and its bound."""
    a = x.double()
    rms = torch.sqrt((a * a).mean(-1, keepdim=True) + eps)
    y = a / rms * w.double()
    return y, 64 * 2.0 ** -24 * y.abs() + 2.0 ** -150 / rms


@pytest.mark.parametrize("K", [640, 4096, 14336, 16512])
@pytest.mark.parametrize("M", [3, 1500])
def test_norm_with_blocks_far_apart(M, K):
    """One block near 2^60, others from 2^-60 down: their y lies between 2^-117 and nothing."""
    dev = need_gpu()
    if M > 3 and K > 4096:
        M = 500
    x = syn.activations(M, K, K, device=dev).float()
    x[:, :128] *= 2.0 ** 60
    for g in range(1, K // 128):
        x[:, 128 * g:128 * g + 128] *= 2.0 ** -(60 + g % 36)
    x = x.to(torch.bfloat16)
    w = (1 + 0.1 * syn.activations(1, K, 5, device=dev).float()).to(torch.bfloat16).view(K)
    st = status(dev)
    xq, sa, _, _ = q.rmsnorm_fp8_block(x, w, EPS, dev_status=st)
    assert read_status(st) == 0
    ref, d = (t.view(M, K // 128, 128) for t in norm_ref(x, w, EPS))
    assert ((sa > 0) & (sa < 2.0 ** -126)).any() and (K == 640 or (sa == 0).any() and ((sa > 0) & (sa < 2.0 ** -140)).any())
    check(xq.view(F8).view(M, K // 128, 128), sa.double().t(), ref, d)


def test_norm_of_a_block_near_2_to_the_100_and_one_near_2_to_the_minus_60():
    dev = need_gpu()
    x = syn.activations(4, 512, 1, device=dev).float()
    x[:, :128] *= 2.0 ** 100
    x[:, 128:] *= 2.0 ** -60
    x = x.to(torch.bfloat16)
    xq, sa, _, _ = q.rmsnorm_fp8_block(x, torch.ones(512, dtype=torch.bfloat16, device=dev), EPS)
    assert torch.all(sa[0] > 0) and not sa[1:].any() and not xq[:, 128:].any() and xq[:, :128].any()


@pytest.mark.parametrize("K", [256, 4096, 32768])
@pytest.mark.parametrize("scale", [2.0 ** -20, 2.0 ** -30, 2.0 ** -36, 2.0 ** -50])
def test_norms_with_small_weights(K, scale):
    """Rows far below the root of eps and weights of 2^-100 (some subnormal): all of y is subnormal, or 0."""
    dev = need_gpu()
    x = (syn.activations(5, K, 3, device=dev).float() * scale).to(torch.bfloat16)
    w = (syn.activations(1, K, 4, device=dev).float() * 2.0 ** -100).to(torch.bfloat16).view(K)
    ref, d = norm_ref(x, w, EPS)
    st = status(dev)
    xq, sa, _, _ = q.rmsnorm_fp8_block(x, w, EPS, dev_status=st)
    assert read_status(st) == 0
    check(xq.view(F8).view(5, K // 128, 128), sa.double().t(), ref.view(5, K // 128, 128), d.view(5, K // 128, 128))


@pytest.mark.parametrize("K", [256, 4096, 32768])
def test_norms_whose_scale_is_nothing(K):
    """Products h w of a few times 2^-149, an eps that leaves them so: scales of 0 and codes of 0, of rows and of blocks."""
    dev = need_gpu()
    x = (syn.activations(5, K, 3, device=dev).float() * 2.0 ** -46).to(torch.bfloat16)
    w = (syn.activations(1, K, 4, device=dev).float() * 2.0 ** -101).to(torch.bfloat16).view(K)
    for call in (q.rmsnorm_fp8, q.rmsnorm_fp8_block):
        st = status(dev)
        xq, sa, _, _ = call(x, w, 1.0, dev_status=st)
        assert read_status(st) == 0 and not sa.any() and not xq.any()


@pytest.mark.parametrize("M", [1, 20, 40, 64, 300])
def test_gated(M):
    """Small codes times scales that are powers of two (every product of them is exact): u and h from 2^-115 down."""
    dev = need_gpu()
    N, K = 256, 256
    xq, _ = q.quant_act_fp8_block(syn.activations(M, K, 1, device=dev))
    wg, _ = q.quant_weights_fp8_block((syn.activations(N, K, 2, device=dev).float()).to(torch.float16))
    g = torch.Generator(device=dev).manual_seed(3)
    wu = torch.randint(0, 3, (N, K), generator=g, device=dev, dtype=torch.uint8) * (torch.rand((N, K), generator=g, device=dev) < 0.02)
    sa = torch.exp2(-3.0 * (torch.arange(M, device=dev) % 5)).expand(K // 128, M).contiguous()
    sg = torch.full((N // 128, K // 128), 2.0 ** -18, device=dev)
    su = torch.full((N // 128, K // 128), 2.0 ** -126, device=dev)
    su[1:] = 2.0 ** -115
    st = status(dev)
    hq, sh, _ = q.gated_fp8_block(xq, sa, wg, sg, wu, su, dev_status=st)
    assert read_status(st) == 0
    xv, gv, uv = act_values(xq, sa), weight_values(wg, sg), weight_values(wu, su)
    ref, d = gated(xv, gv, uv)
    gate = xv @ gv.t()
    # (sums, products and the bound's 2^-118 |u| beside it: nothing here is below g = -87; each subnormal u or h is off by 2^-149)
    d = d - 2.0 ** -118 * (xv @ uv.t()).abs() + 2.0 ** -148 * ((gate * torch.sigmoid(gate)).abs() + 1)
    assert float(gate.min()) > -80 and ((sh > 0) & (sh < (2.0 ** -130 if M == 1 else 2.0 ** -145))).any()
    check(hq.view(F8).view(M, N // 128, 128), sh.double().t(), ref.view(M, N // 128, 128), d.view(M, N // 128, 128))
