"""Products with block scales where the product of a token's scale and a weight's leaves fp32's normal range: what the
header states.  s = sa sw is rounded to fp32 first.  Below 2^-126 that is off by 2^-150 at most, so that to blockref.py's
bound comes, for each block, 2^-150 times the sum of its codes' products in magnitude."""
import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q, synthetic as syn
from blockref import F8, act_values, check_bf16, check_codes, gated, product, weight_values
from gpuhelp import need_gpu, read_status, status

pytestmark = pytest.mark.gpu

# every width of the few-token kernel, whole and in parts of K; the many-token kernel in one round, in parts, and with both
SHAPES = [(1, 128, 512), (5, 300, 2048), (17, 384, 1024), (40, 256, 4096), (70, 300, 512), (128, 384, 2048), (129, 512, 384),
          (300, 640, 4096), (520, 1152, 2048), (2500, 2560, 256)]


def acts(M, K, seed, dev):
    return syn.activations(M, K, seed, device=dev).float()


def parent(N, K, seed, dev, std=0.03):
    return (syn.activations(N, K, seed, device=dev).float() * std).to(torch.float16)


def lost(xq, w8):
    """2^-150 times the sums of the codes' products in magnitude."""
    return 2.0 ** -150 * (xq.view(F8).double().abs() @ w8.view(F8).double().abs().t())


def check(y, xq, sa, w8, sw):
    ref, d = product(act_values(xq, sa), weight_values(w8, sw))
    d = d + lost(xq, w8)
    assert torch.all((y.double() - ref).abs() <= d + 2.0 ** -8 * (ref.abs() + d) + 2.0 ** -134)


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("scale", [2.0 ** -100, 2.0 ** -105, 2.0 ** -120, 2.0 ** -126])
def test_small_activations(M, N, K, scale):
    dev = need_gpu()
    xq, sa = q.quant_act_fp8_block((acts(M, K, M, dev) * scale).to(torch.bfloat16))
    w8, sw = q.quant_weights_fp8_block(parent(N, K, N, dev))
    st = status(dev)
    y = q.linear_fp8_block(xq, sa, w8, sw, dev_status=st)
    assert read_status(st) == 0 and torch.all(torch.isfinite(y))
    check(y, xq, sa, w8, sw)
    if scale == 2.0 ** -100:                              # every product is a normal number: nothing is lost
        s = sa.double().t()[:, None, :] * sw.double().repeat_interleave(128, 0)[None, :N]
        assert s[s > 0].min() >= 2.0 ** -126
        ref, d = product(act_values(xq, sa), weight_values(w8, sw))
        assert torch.all((y.double() - ref).abs() <= d + 2.0 ** -8 * (ref.abs() + d))


@pytest.mark.parametrize("M,N,K", SHAPES)
def test_tokens_of_all_magnitudes(M, N, K):
    """From 2^0 down to 2^-128 beside one another; an ordinary token keeps the bits it has among ordinary ones."""
    dev = need_gpu()
    x = acts(M, K, M + 1, dev)
    plain = x.to(torch.bfloat16)
    order = (torch.arange(M, device=dev) + 1) % 9
    x = (x * torch.exp2(-16.0 * order)[:, None]).to(torch.bfloat16)
    w8, sw = q.quant_weights_fp8_block(parent(N, K, N, dev))
    xq, sa = q.quant_act_fp8_block(x)
    st = status(dev)
    y = q.linear_fp8_block(xq, sa, w8, sw, dev_status=st)
    assert read_status(st) == 0
    check(y, xq, sa, w8, sw)
    want, same = q.linear_fp8_block(*q.quant_act_fp8_block(plain), w8, sw), order == 0
    assert torch.equal(y[same], want[same])


@pytest.mark.parametrize("M,N,K", [(M, -(-N // 128) * 128, K) for M, N, K in SHAPES])
def test_gated(M, N, K):
    """Scales of tokens at 2^-130, the gate's weights' so large that its sums are ordinary ones: u loses what is stated,
    and h that times |silu(g)|."""
    dev = need_gpu()
    xq, _ = q.quant_act_fp8_block(acts(M, K, 1, dev).to(torch.bfloat16))
    wg, wu = (q.quant_weights_fp8_block(parent(N, K, s, dev))[0] for s in (2, 5))

    def scales(rows, cols, top, seed):
        g = torch.Generator(device=dev).manual_seed(seed)
        return (1.0 + torch.rand((rows, cols), generator=g, device=dev)) * top

    sa, sg, su = scales(K // 128, M, 2.0 ** -130, 3), scales(N // 128, K // 128, 2.0 ** 120, 4), scales(N // 128, K // 128, 2.0 ** -10, 6)
    st = status(dev)
    hq, sh, h = q.gated_fp8_block(xq, sa, wg, sg, wu, su, want_bf16=True, dev_status=st)
    assert read_status(st) == 0
    xv, gv, uv = act_values(xq, sa), weight_values(wg, sg), weight_values(wu, su)
    ref, d = gated(xv, gv, uv)
    g = xv @ gv.t()
    a, da = (g * torch.sigmoid(g)).abs(), 1.1 * product(xv, gv)[1]
    d = d + (a + da) * lost(xq, wu) * 1.01
    check_codes(hq, sh, ref, d)
    check_bf16(h, ref, d)
