"""Residual + RMSNorm + E4M3 with a scale for each block of 128 (qspec_rmsnorm_fp8_block) against the formula in 64 bits.

Tolerances are those of the norm with a scale per token: 64 x 2^-24 on the scales; half an E4M3 step (2^-4 of the value,
2^-10 below 2^-6) plus 2^-20 on a code; half a bf16 step plus 2^-20 on y.  h is one fp32 sum rounded to bf16: exact."""
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
    M, K = a.shape
    ref = a / torch.sqrt((a * a).mean(-1, keepdim=True) + eps) * w.double()
    blocks = ref.view(M, K // 128, 128)
    want = blocks.abs().amax(-1) / 448.0
    assert torch.all((sa.double().t() - want).abs() <= 64 * 2.0 ** -24 * want + 2e-45)
    v = blocks / torch.where(want > 0, want, torch.ones_like(want))[..., None]
    code = xq.view(torch.float8_e4m3fn).double().view(M, K // 128, 128)
    assert torch.all((code - v).abs() <= torch.clamp(v.abs() * 2.0 ** -4, min=2.0 ** -10) + v.abs() * 2.0 ** -20)
    if y is not None:
        assert torch.all((y.double() - ref).abs() <= ref.abs() * (2.0 ** -8 + 2.0 ** -20) + 1e-40)


def weights(K, dev):
    return (1 + 0.1 * syn.activations(1, K, 5, device=dev).float()).to(torch.bfloat16).view(K)


@pytest.mark.parametrize("M,K", [(1, 128), (3, 384), (7, 1024), (5, 1152), (1, 4096), (33, 3584), (2, 8192), (3, 14336),
                                 (2, 16512), (1, 32768), (257, 640)])
@pytest.mark.parametrize("residual", [False, True])
def test_against_64_bits(M, K, residual):
    dev = need_gpu()
    x = syn.activations(M, K, M + K, device=dev, outlier_frac=0.01)
    r = syn.activations(M, K, M + K + 1, device=dev, std=2.0) if residual else None
    w = weights(K, dev)
    if M > 2:
        x[1] = 0.0
        x[2, :128] = 0.0
        if residual:
            r[1] = 0.0
            r[2, :128] = 0.0
    st = status(dev)
    got = q.rmsnorm_fp8_block(x, w, EPS, residual=r, want_bf16=True, dev_status=st)
    assert read_status(st) == 0
    check(x, w, EPS, r, got)
    if M > 2:
        assert not got[0][1].any() and not got[1][:, 1].any() and not got[0][2, :128].any() and float(got[1][0, 2]) == 0
    again = q.rmsnorm_fp8_block(x, w, EPS, residual=r)
    assert again[3] is None and torch.equal(again[0], got[0]) and torch.equal(again[1], got[1])


@pytest.mark.parametrize("K", [1152, 2048, 4096, 4224, 8192, 8320, 14336, 16384])
@pytest.mark.parametrize("residual", [False, True])
def test_many_rows_have_the_bits_of_few(K, residual):
    """Above some number of rows a row is spread over half the threads: against 64 bits, and bit by bit against the same
    rows in calls of 40, rows among them whose squares, or whose products with the weights, pass fp32."""
    dev = need_gpu()
    M = 1321
    x = syn.activations(M, K, K, device=dev).float()
    x[1::7] *= 2.0 ** 66
    x[2::7, :128] *= 2.0 ** 100
    x[3] = 0.0
    x = x.to(torch.bfloat16)
    r = syn.activations(M, K, K + 1, device=dev) if residual else None
    w = syn.activations(1, K, 9, device=dev).float().view(K)
    w[128:256] *= 2.0 ** 60
    w = w.to(torch.bfloat16)
    st = status(dev)
    got = q.rmsnorm_fp8_block(x, w, EPS, residual=r, want_bf16=True, dev_status=st)
    assert read_status(st) == 0
    check(x, w, EPS, r, got)
    for m in range(0, M, 40):
        few = q.rmsnorm_fp8_block(x[m:m + 40], w, EPS, residual=None if r is None else r[m:m + 40], want_bf16=True)
        assert torch.equal(few[0], got[0][m:m + 40]) and torch.equal(few[1], got[1][:, m:m + 40])
        assert torch.equal(few[3], got[3][m:m + 40]) and (r is None or torch.equal(few[2], got[2][m:m + 40]))


def test_strided_rows_scales_apart_and_the_residual_in_place():
    dev = need_gpu()
    M, K, lds = 9, 512, 13
    wide = syn.activations(M, 3 * K, 3, device=dev)
    x = wide[:, K:2 * K]
    stream = syn.activations(M, K + 64, 4, device=dev)
    keep = stream.clone()
    w = syn.activations(1, K, 6, device=dev).view(K)
    xq = torch.empty((M, K), dtype=torch.uint8, device=dev)
    sa = torch.full((K // 128, lds), -7.0, device=dev)
    y = torch.full((M, K + 8), 7.0, dtype=torch.bfloat16, device=dev)
    st = status(dev)
    rc = q.qspec_rmsnorm_fp8_block(x, 3 * K, stream, K + 64, w, EPS, M, K, stream, K + 64, xq, sa, lds, y, K + 8, st)
    assert rc == 0 and read_status(st) == 0
    assert torch.equal(stream[:, K:], keep[:, K:]) and torch.all(y[:, K:] == 7.0) and torch.all(sa[:, M:] == -7.0)
    check(x, w, EPS, keep[:, :K], (xq, sa[:, :M], stream[:, :K], y[:, :K]))


@pytest.mark.parametrize("K", [256, 4096, 32768])
@pytest.mark.parametrize("scale", [2.0 ** 100, 2.0 ** 60, 2.0 ** -30])
def test_large_and_small_magnitudes(scale, K):
    dev = need_gpu()
    x = (syn.activations(4, K, 8, device=dev).float() * scale).to(torch.bfloat16)
    w = syn.activations(1, K, 9, device=dev).view(K)
    st = status(dev)
    got = q.rmsnorm_fp8_block(x, w, EPS, want_bf16=True, dev_status=st)
    assert read_status(st) == 0
    check(x, w, EPS, None, got)


@pytest.mark.parametrize("K", [256, 4096])
def test_blocks_of_very_different_magnitudes(K):
    """Products that pass fp32 in one block, and squares that pass it in one row: the other blocks keep their digits."""
    dev = need_gpu()
    x = syn.activations(5, K, 8, device=dev).float()
    w = syn.activations(1, K, 9, device=dev).float().view(K)
    x[1:3, :128] *= 2.0 ** 66                              # squares pass fp32, products do not
    w[128:256] *= 2.0 ** 100
    x[3, 128:256] *= 2.0 ** 40                             # products pass it, squares do not
    x[4, :256] *= 2.0 ** 66                                # both
    x, w = x.to(torch.bfloat16), w.to(torch.bfloat16)
    st = status(dev)
    got = q.rmsnorm_fp8_block(x, w, EPS, want_bf16=True, dev_status=st)
    assert read_status(st) == 0
    check(x, w, EPS, None, got)


def test_weights_of_zero():
    dev = need_gpu()
    x = syn.activations(5, 768, 1, device=dev)
    w = torch.zeros(768, dtype=torch.bfloat16, device=dev)
    st = status(dev)
    xq, sa, _, y = q.rmsnorm_fp8_block(x, w, 1e-30, want_bf16=True, dev_status=st)
    assert read_status(st) == 0 and not sa.any() and not xq.any() and not y.any()


@pytest.mark.parametrize("where", ["x", "residual", "w"])
@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("K", [384, 4096])
def test_non_finite_inputs_are_flagged(where, value, K):
    dev = need_gpu()
    t = {"x": syn.activations(3, K, 1, device=dev), "residual": syn.activations(3, K, 2, device=dev),
         "w": syn.activations(1, K, 3, device=dev)}
    t[where][-1, 77] = value
    st = status(dev)
    xq, sa, h, _ = q.rmsnorm_fp8_block(t["x"], t["w"].view(K), EPS, residual=t["residual"], dev_status=st)
    assert read_status(st) == q.ERR_NONFINITE
    if where != "w":                    # the other rows are what they were
        check(t["x"][:2], t["w"].view(K), EPS, t["residual"][:2], (xq[:2], sa[:, :2], h[:2], None))
