"""Residual + RMSNorm + E4M3 (qspec_rmsnorm_fp8) against the formula in 64 bits.

Tolerances.  The sum of squares takes at most 32 fused steps in a thread and
ten levels of a tree (42 x 2^-24 relative, all terms positive), half of it
after the root; root, division and products add a few roundings: 64 x 2^-24 on
the scales.  A code is off the 64-bit quotient by half an E4M3 step (2^-4 of
the value, 2^-10 below 2^-6) plus fp32 roundings (2^-20 covers them); y by
half a bf16 step (2^-8) plus the same.  h is one fp32 sum rounded to bf16:
exact."""
import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q, synthetic as syn
from gpuhelp import need_gpu, read_status, status

pytestmark = pytest.mark.gpu
EPS = 1e-5


def check(x, w, eps, r, got):
    xq, sa, h, y = got
    hh = x.float()
    if r is not None:
        hh = (x.float() + r.float()).to(torch.bfloat16)
        assert torch.equal(h, hh)
    a = hh.double()
    ref = a / torch.sqrt((a * a).mean(-1, keepdim=True) + eps) * w.double()
    ref_sa = ref.abs().amax(-1) / 448.0
    assert torch.all((sa.double() - ref_sa).abs() <= 64 * 2.0 ** -24 * ref_sa + 1e-45)
    v = torch.where(ref_sa[:, None] > 0, ref / ref_sa[:, None], torch.zeros_like(ref))
    code = xq.view(torch.float8_e4m3fn).double()
    assert torch.all((code - v).abs() <= torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10) + v.abs() * 2.0 ** -20)
    if y is not None:
        assert torch.all((y.double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -20) + 1e-40)


@pytest.mark.parametrize("M,K", [(1, 128), (3, 384), (7, 1024), (5, 1152), (1, 4096), (33, 3584), (2, 8192),
                                 (3, 14336), (2, 16512), (1, 32768), (257, 640)])
@pytest.mark.parametrize("residual", [False, True])
def test_against_64_bits(M, K, residual):
    dev = need_gpu()
    x = syn.activations(M, K, M + K, device=dev, outlier_frac=0.01)
    r = syn.activations(M, K, M + K + 1, device=dev, std=2.0) if residual else None
    w = (1 + 0.1 * syn.activations(1, K, 5, device=dev).float()).to(torch.bfloat16).view(K)
    if M > 2:
        x[1] = 0.0
        if residual:
            r[1] = 0.0
    st = status(dev)
    got = q.rmsnorm_fp8(x, w, EPS, residual=r, want_bf16=True, dev_status=st)
    assert read_status(st) == 0
    check(x, w, EPS, r, got)
    if M > 2:
        assert float(got[1][1]) == 0.0 and int(got[0][1].sum()) == 0
    # the same codes without the bf16 output, and what the Q8 quantiser makes of the same rows is as near
    again = q.rmsnorm_fp8(x, w, EPS, residual=r)
    assert again[3] is None and torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


def test_strided_rows_and_the_residual_in_place():
    dev = need_gpu()
    M, K = 9, 512
    wide = syn.activations(M, 3 * K, 3, device=dev)
    x = wide[:, K:2 * K]
    stream = syn.activations(M, K + 64, 4, device=dev)
    keep = stream.clone()
    w = syn.activations(1, K, 6, device=dev).view(K)
    xq = torch.empty((M, K), dtype=torch.uint8, device=dev)
    sa = torch.empty(M, dtype=torch.float32, device=dev)
    y = torch.full((M, K + 8), 7.0, dtype=torch.bfloat16, device=dev)
    st = status(dev)
    rc = q.qspec_rmsnorm_fp8(x, 3 * K, stream, K + 64, w, EPS, M, K, stream, K + 64, xq, sa, y, K + 8, st)
    assert rc == 0 and read_status(st) == 0
    assert torch.equal(stream[:, K:], keep[:, K:]) and torch.all(y[:, K:] == 7.0)
    check(x, w, EPS, keep[:, :K], (xq, sa, stream[:, :K], y[:, :K]))


@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** 60, 2.0 ** -30, 2.0 ** -100, 2.0 ** -126])
@pytest.mark.parametrize("K", [256, 4096])
def test_extreme_magnitudes(scale, K):
    dev = need_gpu()
    x = (syn.activations(4, K, 8, device=dev).float() * scale).to(torch.bfloat16)
    w = syn.activations(1, K, 9, device=dev).view(K)
    st = status(dev)
    got = q.rmsnorm_fp8(x, w, EPS, want_bf16=True, dev_status=st)
    assert read_status(st) == 0
    if scale > 1e-20:
        check(x, w, EPS, None, got)
    else:                               # codes do not depend on the norm; the scale may be a subnormal
        p = x.double() * w.double()
        v = p / p.abs().amax(-1, keepdim=True) * 448.0
        code = got[0].view(torch.float8_e4m3fn).double()
        # products below 2^-126 lose bits: 2^-149 absolute
        lost = 448.0 * 2.0 ** -149 / p.abs().amax(-1, keepdim=True)
        assert torch.all((code - v).abs() <= torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10)
                         + v.abs() * 2.0 ** -20 + 2 * lost * (1 + v.abs()))


def test_small_eps_and_weights_of_zero():
    dev = need_gpu()
    x = syn.activations(5, 768, 1, device=dev)
    w = torch.zeros(768, dtype=torch.bfloat16, device=dev)
    st = status(dev)
    xq, sa, _, y = q.rmsnorm_fp8(x, w, 1e-30, want_bf16=True, dev_status=st)
    assert read_status(st) == 0
    assert torch.all(sa == 0) and torch.all(xq == 0) and torch.all(y == 0)


@pytest.mark.parametrize("where", ["x", "residual", "w"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("K", [384, 4096])
def test_non_finite_inputs_are_flagged(where, value, K):
    dev = need_gpu()
    t = {"x": syn.activations(3, K, 1, device=dev), "residual": syn.activations(3, K, 2, device=dev),
         "w": syn.activations(1, K, 3, device=dev)}
    t[where][-1, 77] = value
    st = status(dev)
    xq, sa, h, _ = q.rmsnorm_fp8(t["x"], t["w"].view(K), EPS, residual=t["residual"], dev_status=st)
    assert read_status(st) == q.ERR_NONFINITE
    if where != "w":                    # the other rows are what they were
        check(t["x"][:2], t["w"].view(K), EPS, t["residual"][:2], (xq[:2], sa[:2], h[:2], None))


def test_feeds_the_fp8_linear():
    dev = need_gpu()
    M, N, K = 5, 384, 1024
    x, r = syn.activations(M, K, 1, device=dev), syn.activations(M, K, 2, device=dev)
    w = syn.activations(1, K, 3, device=dev).view(K)
    w8, s8 = q.quant_weights_fp8((syn.activations(N, K, 4, device=dev).float() * 0.02).to(torch.float16))
    xq, sa, _, _ = q.rmsnorm_fp8(x, w, EPS, residual=r)
    y = q.linear_fp8(xq, sa, w8, s8)
    ref = ((xq.view(torch.float8_e4m3fn).double() @ w8.view(torch.float8_e4m3fn).double().T)
           * sa.double()[:, None] * s8.double())
    assert torch.all((y.double() - ref).abs() <= 1e-2 * (1 + ref.abs()))     # the linear's own bound


@pytest.mark.parametrize("K", [256, 4096, 32768])
def test_large_magnitudes_with_a_residual(K):
    """Squares that pass fp32 in some rows: those rows are read again from the sum that was written."""
    dev = need_gpu()
    x = syn.activations(5, K, 8, device=dev).float()
    x[1:3] *= 2.0 ** 90
    x = x.to(torch.bfloat16)
    r = (syn.activations(5, K, 10, device=dev).float() * 2.0 ** 89).to(torch.bfloat16)
    r[0] = syn.activations(1, K, 11, device=dev)[0]
    w = syn.activations(1, K, 9, device=dev).view(K)
    st = status(dev)
    got = q.rmsnorm_fp8(x, w, EPS, residual=r, want_bf16=True, dev_status=st)
    assert read_status(st) == 0
    check(x, w, EPS, r, got)
