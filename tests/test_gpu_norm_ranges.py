"""Residual + RMSNorm + E4M3 at the ends of the number range: products h w past fp32 where y is not, and y past bf16.

Tolerances as for the ordinary rows: 64 x 2^-24 on the scales, half an E4M3 step on the codes, half a bf16 step on y,
2^-20 for the fp32 roundings."""
import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q
from gpuhelp import need_gpu, read_status, status

pytestmark = pytest.mark.gpu
EPS = 1e-5


def check(x, w, eps, got):
    xq, sa, _, y = got
    a = x.double()
    ref = a / torch.sqrt((a * a).mean(-1, keepdim=True) + eps) * w.double()
    ref_sa = ref.abs().amax(-1) / 448.0
    assert torch.all((sa.double() - ref_sa).abs() <= 64 * 2.0 ** -24 * ref_sa)
    v = ref / ref_sa[:, None]
    code = xq.view(torch.float8_e4m3fn).double()
    assert torch.all((code - v).abs() <= torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10) + v.abs() * 2.0 ** -20)
    assert torch.all((y.double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -20) + 1e-40)


@pytest.mark.parametrize("K", [128, 896, 4096, 14336])
@pytest.mark.parametrize("h,w", [(100.0, 1e37), (30.0, 2e37), (1e5, 1e35), (1e10, 1e30), (1e25, 1e20), (1e19, 1.0)])
def test_products_past_fp32(K, h, w):
    """h w passes 3.4e38, y = h w rstd does not; with |h| around and above 1e19 the squares pass it too."""
    dev = need_gpu()
    g = torch.Generator(device=dev).manual_seed(K)
    x = (h * (0.5 + torch.rand((3, K), generator=g, device=dev, dtype=torch.float64))).to(torch.bfloat16)
    x[1] = -x[1]
    x[2] = torch.randn(K, generator=g, device=dev).to(torch.bfloat16)         # an ordinary row next to them
    ww = torch.full((K,), w, device=dev).to(torch.bfloat16)
    if w > 1e36:
        ww[::2] = 1.0                                                         # (and small products among large ones)
        x[2] *= 0.01
    st = status(dev)
    got = q.rmsnorm_fp8(x, ww, EPS, want_bf16=True, dev_status=st)
    assert read_status(st) == 0
    check(x, ww, EPS, got)


@pytest.mark.parametrize("K", [128, 4096])
def test_y_past_bf16(K):
    """A y between the largest bf16 value and fp32's is finite for the codes; as a bf16 output it is inf, and flagged."""
    dev = need_gpu()
    x = torch.ones((1, K), device=dev)
    x[0, K // 4:] = 1 - 2.0 ** -8                              # x / rms = 1.0029 where x = 1
    w = torch.ones(K, device=dev)
    w[0] = torch.finfo(torch.bfloat16).max                     # y = 1.0029 x 3.3895e38: past the midpoint 3.3962e38
    x, w = x.to(torch.bfloat16), w.to(torch.bfloat16)
    st = status(dev)
    xq, sa, _, _ = q.rmsnorm_fp8(x, w, EPS, dev_status=st)
    assert read_status(st) == 0 and torch.isfinite(sa).all() and int(xq[0, 0]) == 0x7E
    _, _, _, y = q.rmsnorm_fp8(x, w, EPS, want_bf16=True, dev_status=st)
    assert torch.isinf(y[0, 0]) and read_status(st) == q.ERR_NONFINITE
