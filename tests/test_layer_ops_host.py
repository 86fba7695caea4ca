"""Refusals of the norm, 4-bit cache and attention calls: rejected on the host,
before any launch (no GPU needed)."""
import ctypes

import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding
from quantized_speculative_decoding_shared_gb300 import build as qbuild

V = ctypes.c_void_p
NULL, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 5


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return binding.load_library()


def fake(n=0x1000):
    """A non-null, aligned address that the calls below must not touch."""
    return V(n)


def refuse(fn, ok, order, cases):
    for want, change in cases:
        a = dict(ok, **change)
        assert fn(*[a[k] for k in order]) == want, change


def test_rmsnorm_refusals(lib):
    ok = dict(x=fake(), ldx=256, r=fake(), ldr=256, w=fake(), eps=1e-5, M=2, K=256, h=fake(), ldh=256, xq=fake(),
              sa=fake(), y=fake(), ldy=256, st=None, s=None)
    refuse(lib.qspec_rmsnorm_fp8, ok, list(ok), [
        (NULL, dict(x=None)), (NULL, dict(w=None)), (NULL, dict(xq=None)), (NULL, dict(sa=None)),
        (NULL, dict(h=None)), (NULL, dict(r=None)),                     # residual and h come together
        (SHAPE, dict(M=0)), (SHAPE, dict(K=0)), (SHAPE, dict(K=200)), (SHAPE, dict(K=32896)),
        (SHAPE, dict(eps=0.0)), (SHAPE, dict(eps=-1.0)), (SHAPE, dict(eps=float("nan"))),
        (SHAPE, dict(eps=float("inf"))), (SHAPE, dict(ldx=248)), (SHAPE, dict(ldr=248)), (SHAPE, dict(ldh=248)),
        (SHAPE, dict(ldy=248)), (ALIGN, dict(ldx=257)), (ALIGN, dict(ldr=260)), (ALIGN, dict(ldh=258)),
        (ALIGN, dict(ldy=260)), (ALIGN, dict(x=fake(0x1008))), (ALIGN, dict(r=fake(0x1002))),
        (ALIGN, dict(w=fake(0x1004))), (ALIGN, dict(h=fake(0x1008))), (ALIGN, dict(xq=fake(0x1004))),
        (ALIGN, dict(sa=fake(0x1002))), (ALIGN, dict(y=fake(0x1008)))])


@pytest.mark.parametrize("load", [False, True])
def test_kv4_rows_refusals(lib, load):
    rows = dict(k=fake(), ldk=256, v=fake(), ldv=256)
    cache = dict(kc=fake(), ks=fake(), vc=fake(), vs=fake())
    mid = dict(start=fake(), base=fake(), rows=3, B=2, H=2, T=16, D=128)
    ok = dict(cache, **mid, **rows, st=None, s=None) if load else dict(rows, **mid, **cache, st=None, s=None)
    refuse(lib.qspec_kv4_load if load else lib.qspec_kv4_append, ok, list(ok), [
        (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(start=None)), (NULL, dict(base=None)),
        (NULL, dict(kc=None)), (NULL, dict(ks=None)), (NULL, dict(vc=None)), (NULL, dict(vs=None)),
        (SHAPE, dict(rows=-1)), (SHAPE, dict(B=0)), (SHAPE, dict(H=0)), (SHAPE, dict(T=0)), (SHAPE, dict(D=96)),
        (SHAPE, dict(D=256)), (SHAPE, dict(ldk=248)), (SHAPE, dict(ldv=248)), (ALIGN, dict(ldk=260)),
        (ALIGN, dict(ldv=257)), (ALIGN, dict(k=fake(0x1008))), (ALIGN, dict(v=fake(0x1002))),
        (ALIGN, dict(kc=fake(0x1008))), (ALIGN, dict(vc=fake(0x1004))), (ALIGN, dict(ks=fake(0x1002))),
        (ALIGN, dict(vs=fake(0x1001))), (ALIGN, dict(start=fake(0x1002))), (ALIGN, dict(base=fake(0x1001)))])


def test_attn_kv4_refusals(lib):
    need = binding.qspec_attn_kv4_workspace_bytes(2, 5, 8, 2, 128)
    assert need > 0 and need % 16 == 0
    ok = dict(q=fake(), ldq=1024, kc=fake(), ks=fake(), vc=fake(), vs=fake(), n=fake(), B=2, R=5, Hq=8, H=2, T=64,
              D=128, scale=0.1, o=fake(), ldo=1024, ws=fake(), wsb=need, st=None, s=None)
    refuse(lib.qspec_attn_kv4, ok, list(ok), [
        (NULL, dict(q=None)), (NULL, dict(kc=None)), (NULL, dict(ks=None)), (NULL, dict(vc=None)),
        (NULL, dict(vs=None)), (NULL, dict(n=None)), (NULL, dict(o=None)), (NULL, dict(ws=None)),
        (SHAPE, dict(B=0)), (SHAPE, dict(R=0)), (SHAPE, dict(R=18)), (SHAPE, dict(Hq=7)), (SHAPE, dict(H=0)),
        (SHAPE, dict(Hq=1)), (SHAPE, dict(T=0)), (SHAPE, dict(D=80)), (SHAPE, dict(scale=float("nan"))),
        (SHAPE, dict(ldq=1016)), (SHAPE, dict(ldo=1016)), (ALIGN, dict(ldq=1025)), (ALIGN, dict(ldo=1028)),
        (ALIGN, dict(q=fake(0x1008))), (ALIGN, dict(o=fake(0x1008))), (ALIGN, dict(kc=fake(0x1008))),
        (ALIGN, dict(vc=fake(0x1008))), (ALIGN, dict(ks=fake(0x1002))), (ALIGN, dict(vs=fake(0x1002))),
        (ALIGN, dict(n=fake(0x1002))), (ALIGN, dict(ws=fake(0x1008))), (WORKSPACE, dict(wsb=need - 1))])
    for bad in ((0, 1, 8, 2, 128), (1, 18, 8, 2, 128), (1, 1, 7, 2, 128), (1, 1, 8, 2, 96)):
        assert binding.qspec_attn_kv4_workspace_bytes(*bad) == 0


def test_attn_prompt_refusals(lib):
    ok = dict(q=fake(), ldq=1024, k=fake(), ldk=256, v=fake(), ldv=256, qs=fake(), ks=fake(), qr=10, kr=12, B=2, Hq=8,
              H=2, D=128, scale=0.1, o=fake(), ldo=1024, st=None, s=None)
    refuse(lib.qspec_attn_prompt, ok, list(ok), [
        (NULL, dict(q=None)), (NULL, dict(k=None)), (NULL, dict(v=None)), (NULL, dict(qs=None)),
        (NULL, dict(ks=None)), (NULL, dict(o=None)), (SHAPE, dict(qr=-1)), (SHAPE, dict(kr=-1)), (SHAPE, dict(B=0)),
        (SHAPE, dict(H=0)), (SHAPE, dict(Hq=7)), (SHAPE, dict(Hq=1)), (SHAPE, dict(D=32)),
        (SHAPE, dict(scale=float("inf"))), (SHAPE, dict(ldq=1016)), (SHAPE, dict(ldk=248)), (SHAPE, dict(ldv=248)),
        (SHAPE, dict(ldo=1016)), (ALIGN, dict(ldq=1028)), (ALIGN, dict(ldk=257)), (ALIGN, dict(ldv=260)),
        (ALIGN, dict(ldo=1025)), (ALIGN, dict(q=fake(0x1008))), (ALIGN, dict(k=fake(0x1002))),
        (ALIGN, dict(v=fake(0x1004))), (ALIGN, dict(o=fake(0x1008))), (ALIGN, dict(qs=fake(0x1002))),
        (ALIGN, dict(ks=fake(0x1001)))])


def test_conveniences_refuse_what_they_cannot_pass_on():
    x = torch.zeros((2, 256), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.rmsnorm_fp8(x, torch.zeros(256, dtype=torch.bfloat16), 1e-5)          # not on a GPU
    q = torch.zeros((2, 4, 128), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        binding.attn_prompt(q, q, q, torch.zeros(2, dtype=torch.int32))
    cache = binding.kv4_cache(1, 2, 8, 128, device="cpu")
    assert cache[0].shape == (1, 2, 8, 64) and cache[1].shape == (1, 2, 8)
    with pytest.raises(ValueError):
        binding.kv4_append(cache, q, q, torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    with pytest.raises(ValueError):
        binding.attn_kv4(q, cache, torch.zeros(1, dtype=torch.int32), 0.1)


def test_sizes_past_what_the_kernels_count(lib):
    """Row numbers of the cache calls and tile numbers of the attention are 32-bit ones."""
    rows = dict(k=fake(), ldk=256, v=fake(), ldv=256, start=fake(), base=fake(), rows=2 ** 31 - 8, B=2, H=2, T=16, D=128,
                kc=fake(), ks=fake(), vc=fake(), vs=fake(), st=None, s=None)
    refuse(lib.qspec_kv4_append, rows, list(rows), [(SHAPE, {}), (SHAPE, dict(rows=2 ** 30, H=2 ** 12, ldk=2 ** 19, ldv=2 ** 19))])
    need = binding.qspec_attn_kv4_workspace_bytes(1, 1, 8, 2, 128)
    ok = dict(q=fake(), ldq=1024, kc=fake(), ks=fake(), vc=fake(), vs=fake(), len=fake(), B=1, R=1, Hq=8, H=2, T=64, D=128,
              scale=0.1, o=fake(), ldo=1024, ws=fake(), n=need, st=None, s=None)
    refuse(lib.qspec_attn_kv4, ok, list(ok), [(SHAPE, dict(T=2 ** 30 + 1)), (SHAPE, dict(B=64, T=2 ** 30)),
                                              (SHAPE, dict(R=17, Hq=16384, ldq=2 ** 21, ldo=2 ** 21, T=2 ** 28))])
