"""Refusals of the attention kernels' diagnostic entries, before any launch (no GPU needed)."""
import ctypes

import pytest

from quantized_speculative_decoding_shared_gb300 import binding
from quantized_speculative_decoding_shared_gb300 import build as qbuild

NULL, SHAPE, ALIGN, WORKSPACE = 1, 2, 3, 5


@pytest.fixture(scope="module")
def lib():
    qbuild.build()
    return binding.load_library()


def fake(n=0x1000):
    return ctypes.c_void_p(n)


def test_refusals(lib):
    need = binding.qspec_attn_kv4_workspace_bytes(2, 5, 8, 2, 128)
    kv4 = dict(q=fake(), ldq=1024, kc=fake(), ks=fake(), vc=fake(), vs=fake(), n=fake(), B=2, R=5, Hq=8, H=2, T=64, D=128, scale=0.1,
               o=fake(), ldo=1024, ws=fake(), wsb=need, limit=1000, stall=1, st=None, s=None)
    prompt = dict(q=fake(), ldq=1024, k=fake(), ldk=256, v=fake(), ldv=256, qs=fake(), ks=fake(), qr=10, kr=12, B=2, Hq=8, H=2, D=128,
                  scale=0.1, o=fake(), ldo=1024, limit=1000, stall=1, st=None, s=None)
    for fn, ok, cases in (
            (lib.qspec_debug_attn_kv4_bounded, kv4, [(SHAPE, dict(limit=0)), (NULL, dict(ws=None)), (SHAPE, dict(R=18)),
                                                     (ALIGN, dict(q=fake(0x1008))), (WORKSPACE, dict(wsb=need - 1))]),
            (lib.qspec_debug_attn_prompt_bounded, prompt, [(SHAPE, dict(limit=0)), (NULL, dict(q=None)), (SHAPE, dict(D=32)),
                                                           (ALIGN, dict(ldk=257))])):
        for want, change in cases:
            a = dict(ok, **change)
            assert fn(*a.values()) == want, change
