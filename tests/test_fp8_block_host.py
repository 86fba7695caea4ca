"""Refusals of the E4M3 calls with block scales: on the host, before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding
from quantized_speculative_decoding_shared_gb300 import build as qbuild

V = ctypes.c_void_p
NULL, SHAPE, ALIGN = 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return binding.load_library()


def at(n=0x1000):
    """An aligned address that the calls must not touch."""
    return V(n)


def refuse(fn, ok, cases):
    for want, change in cases:
        a = dict(ok, **change)
        assert fn(*a.values()) == want, change


def test_quantisers(lib):
    refuse(lib.qspec_quant_weights_fp8_block, dict(w=at(), N=3, K=256, w8=at(), sw=at(), st=None, s=None), [
        (NULL, dict(w=None)), (NULL, dict(w8=None)), (NULL, dict(sw=None)), (SHAPE, dict(N=0)), (SHAPE, dict(K=0)),
        (SHAPE, dict(K=200)), (SHAPE, dict(K=-128)), (SHAPE, dict(N=2 ** 31 - 1, K=2 ** 31 - 128)),
        (ALIGN, dict(w=at(0x1008))), (ALIGN, dict(w8=at(0x1004))), (ALIGN, dict(sw=at(0x1002)))])
    refuse(lib.qspec_quant_act_fp8_block, dict(x=at(), M=3, K=256, ldx=256, xq=at(), sa=at(), lds=3, st=None, s=None), [
        (NULL, dict(x=None)), (NULL, dict(xq=None)), (NULL, dict(sa=None)), (SHAPE, dict(M=0)), (SHAPE, dict(K=100)),
        (SHAPE, dict(ldx=248)), (SHAPE, dict(lds=2)), (SHAPE, dict(M=2 ** 31 - 1, lds=2 ** 31 - 1, K=2 ** 31 - 128, ldx=2 ** 31 - 8)),
        (ALIGN, dict(ldx=260)), (ALIGN, dict(x=at(0x1008))), (ALIGN, dict(xq=at(0x1004))), (ALIGN, dict(sa=at(0x1001)))])


def test_norm(lib):
    ok = dict(x=at(), ldx=256, r=at(), ldr=256, w=at(), eps=1e-5, M=2, K=256, h=at(), ldh=256, xq=at(), sa=at(), lds=2,
              y=at(), ldy=256, st=None, s=None)
    refuse(lib.qspec_rmsnorm_fp8_block, ok, [
        (NULL, dict(x=None)), (NULL, dict(w=None)), (NULL, dict(xq=None)), (NULL, dict(sa=None)), (NULL, dict(h=None)),
        (NULL, dict(r=None)), (SHAPE, dict(M=0)), (SHAPE, dict(K=0)), (SHAPE, dict(K=200)), (SHAPE, dict(K=32896)),
        (SHAPE, dict(eps=0.0)), (SHAPE, dict(eps=float("nan"))), (SHAPE, dict(eps=float("inf"))), (SHAPE, dict(lds=1)),
        (SHAPE, dict(ldx=248)), (SHAPE, dict(ldr=248)), (SHAPE, dict(ldh=248)), (SHAPE, dict(ldy=248)),
        (ALIGN, dict(ldx=257)), (ALIGN, dict(ldr=260)), (ALIGN, dict(ldh=258)), (ALIGN, dict(ldy=260)),
        (ALIGN, dict(x=at(0x1008))), (ALIGN, dict(r=at(0x1002))), (ALIGN, dict(w=at(0x1004))), (ALIGN, dict(h=at(0x1008))),
        (ALIGN, dict(xq=at(0x1004))), (ALIGN, dict(sa=at(0x1002))), (ALIGN, dict(y=at(0x1008)))])


def test_linear(lib):
    ok = dict(xq=at(), sa=at(), lds=5, w=at(), sw=at(), M=5, N=100, K=256, y=at(), ldy=100, st=None, s=None)
    refuse(lib.qspec_linear_fp8_block, ok, [
        (NULL, dict(xq=None)), (NULL, dict(sa=None)), (NULL, dict(w=None)), (NULL, dict(sw=None)), (NULL, dict(y=None)),
        (SHAPE, dict(M=0)), (SHAPE, dict(N=0)), (SHAPE, dict(K=0)), (SHAPE, dict(K=130)), (SHAPE, dict(ldy=99)),
        (SHAPE, dict(lds=4)), (SHAPE, dict(M=2 ** 22 + 1, lds=2 ** 23)), (SHAPE, dict(N=2 ** 30 + 1, ldy=2 ** 30 + 1)),
        (ALIGN, dict(xq=at(0x1008))), (ALIGN, dict(w=at(0x1008))), (ALIGN, dict(sa=at(0x1002))),
        (ALIGN, dict(sw=at(0x1002))), (ALIGN, dict(y=at(0x1001)))])


def test_gated(lib):
    ok = dict(xq=at(), sa=at(), lds=5, wg=at(), sg=at(), wu=at(), su=at(), M=5, N=128, K=256, hq=at(), sh=at(), ldh=5,
              h=at(), ldy=128, st=None, s=None)
    refuse(lib.qspec_gated_fp8_block, ok, [
        (NULL, dict(xq=None)), (NULL, dict(sa=None)), (NULL, dict(wg=None)), (NULL, dict(sg=None)), (NULL, dict(wu=None)),
        (NULL, dict(su=None)), (NULL, dict(hq=None)), (NULL, dict(sh=None)), (NULL, dict(hq=None, sh=None, h=None)),
        (SHAPE, dict(M=0)), (SHAPE, dict(N=0)), (SHAPE, dict(N=100)), (SHAPE, dict(N=129)), (SHAPE, dict(K=130)),
        (SHAPE, dict(lds=4)), (SHAPE, dict(ldh=4)), (SHAPE, dict(ldy=127)), (SHAPE, dict(M=2 ** 22 + 1, lds=2 ** 23, ldh=2 ** 23)),
        (ALIGN, dict(xq=at(0x1008))), (ALIGN, dict(wg=at(0x1008))), (ALIGN, dict(wu=at(0x1004))),
        (ALIGN, dict(sa=at(0x1002))), (ALIGN, dict(sg=at(0x1001))), (ALIGN, dict(su=at(0x1002))),
        (ALIGN, dict(hq=at(0x1008))), (ALIGN, dict(sh=at(0x1002))), (ALIGN, dict(h=at(0x1001)))])


def test_conveniences_refuse_what_they_cannot_pass_on():
    x, u8 = torch.zeros((2, 256), dtype=torch.bfloat16), torch.zeros((2, 256), dtype=torch.uint8)
    s = torch.zeros((2, 2))
    for call in (lambda: binding.quant_act_fp8_block(x), lambda: binding.quant_weights_fp8_block(x.to(torch.float16)),
                 lambda: binding.rmsnorm_fp8_block(x, x[0], 1e-5), lambda: binding.linear_fp8_block(u8, s, u8, s),
                 lambda: binding.gated_fp8_block(u8, s, u8, s, u8, s)):
        with pytest.raises(ValueError):
            call()


class OnDevice:
    """A tensor that says it lies on a GPU."""

    def __init__(self, t):
        self.t, self.device = t, torch.device("cuda")

    def __getattr__(self, name):
        return getattr(self.t, name)


def test_rows_of_scales_that_overlap_are_refused():
    xq = OnDevice(torch.zeros((3, 256), dtype=torch.uint8))
    wide = torch.zeros((2, 8))
    assert binding._block_codes(xq, OnDevice(wide[:, :3])) == (3, 256, 8)
    assert binding._block_codes(xq, OnDevice(wide[0, :6].view(2, 3))) == (3, 256, 3)
    one = OnDevice(torch.zeros((1, 256), dtype=torch.uint8))
    assert binding._block_codes(one, OnDevice(wide[:, :1])) == (1, 256, 8)
    block = OnDevice(torch.zeros((3, 128), dtype=torch.uint8))
    assert binding._block_codes(block, OnDevice(wide[:1, :3])) == (3, 128, 3)      # (one row: its distance is nobody's)
    assert binding._block_codes(block, OnDevice(torch.zeros(3).expand(1, 3))) == (3, 128, 3)
    for codes, sa in ((xq, torch.zeros(3).expand(2, 3)), (xq, torch.zeros(6).as_strided((2, 3), (2, 1))),
                      (xq, torch.zeros((3, 2)).t()), (xq, torch.zeros((2, 1)).expand(2, 3)), (one, torch.zeros(1).expand(2, 1)),
                      (xq, torch.zeros(6)), (xq, torch.zeros((2, 4))), (one, torch.empty((2, 1), device="meta").as_strided((2, 1), (2 ** 31, 1)))):
        with pytest.raises(ValueError):
            binding._block_codes(codes, OnDevice(sa))
    far = torch.empty((2, 128), dtype=torch.bfloat16, device="meta").as_strided((2, 128), (2 ** 31 + 128, 1))
    with pytest.raises(ValueError):
        binding._rows_of(OnDevice(far), "x")


def test_the_diagnostic_entry(lib):
    linear = dict(xq=at(), sa=at(), lds=5, w=at(), sw=at(), w1=None, s1=None, M=5, N=100, K=256, hq=None, sh=None, ldh=0, y=at(), ldy=100,
                  limit=1000, stall=1, st=None, s=None)
    refuse(lib.qspec_debug_fp8_block_bounded, linear, [
        (SHAPE, dict(limit=0)), (NULL, dict(y=None)), (SHAPE, dict(K=130)), (SHAPE, dict(lds=4)), (ALIGN, dict(w=at(0x1008)))])
    gated = dict(linear, w1=at(), s1=at(), N=128, hq=at(), sh=at(), ldh=5, ldy=128)
    refuse(lib.qspec_debug_fp8_block_bounded, gated, [
        (SHAPE, dict(limit=0)), (NULL, dict(s1=None)), (NULL, dict(sh=None)), (SHAPE, dict(N=100)), (ALIGN, dict(w1=at(0x1008)))])
