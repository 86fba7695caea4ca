"""The bounded waits of the two attention kernels, tested without any fault.

Through the diagnostic entries the warp that issues the score products waits, with a short bound, on a barrier that
nothing arrives at.  The kernel must give up, walk to its end past every barrier its warps share, let what it has in
flight finish, free its tensor memory, report QSPEC_ERR_TIMEOUT and return; the context stays usable, and for the
cache attention the workspace too: a regular call on the same one then gives the bits of a call on a fresh one."""
import math

import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q
from gpuhelp import need_gpu, read_status, status
from layerref import random_cache
import test_gpu_attn_kv4 as kv4
import test_gpu_attn_prompt as prompt

pytestmark = pytest.mark.gpu

REGULAR = 1 << 22           # the library's own bound
SHORT = 2000                # a bound the stalled wait runs through


# one CTA to a task; parts of one task in many CTAs (whole parts, equal shares); rows in blocks; every width of the
# products; more sequences than a warp has lanes
@pytest.mark.parametrize("B,R,H,G,D,T", [(2, 1, 2, 4, 128, 100), (1, 1, 8, 4, 128, 20000), (3, 9, 4, 7, 128, 3001), (2, 17, 2, 8, 64, 5000),
                                         (16, 5, 8, 4, 128, 1500), (40, 1, 2, 4, 64, 700)])
def test_cache_attention_then_a_regular_call(B, R, H, G, D, T):
    dev = need_gpu()
    lens = [T - 37 * b % T for b in range(B)]
    cache = random_cache(B, H, T, D, 5, dev)
    x = kv4.queries(B * R, H * G, D, 6, dev)
    length, scale, ld = kv4.ints(lens, dev), 1 / math.sqrt(D), H * G * D
    want = q.attn_kv4(x, cache, length, scale)
    ws = q.attn_kv4_workspace(B, R, H * G, H, D)

    def bounded(limit, stall):
        o, st = torch.full_like(x, float("nan")), status(dev)
        rc = q.qspec_debug_attn_kv4_bounded(x, ld, *cache, length, B, R, H * G, H, T, D, scale, o, ld, ws, ws.numel(), limit, stall, st)
        assert rc == q.OK
        torch.cuda.synchronize()                # the kernel returned
        return o, read_status(st)

    for _ in range(2):
        assert bounded(SHORT, 1)[1] == q.ERR_TIMEOUT
        o, st = bounded(REGULAR, 0)
        assert st == 0 and torch.equal(o, want)
    st = status(dev)
    assert torch.equal(q.attn_kv4(x, cache, length, scale, workspace=ws, dev_status=st), want) and read_status(st) == 0
    kv4.check(x, cache, lens, R, scale, want)


@pytest.mark.parametrize("H,G,D,lens", [(1, 1, 64, [5]), (8, 4, 128, [3000]), (4, 7, 128, [700, 1, 350]), (2, 2, 64, [(b * 29) % 67 for b in range(50)])])
def test_prompt_attention_then_a_regular_call(H, G, D, lens):
    dev = need_gpu()
    n, B, scale = sum(lens), len(lens), 1 / math.sqrt(D)
    x, k, v = prompt.heads(n, H * G, D, 1, dev), prompt.heads(n, H, D, 2, dev), prompt.heads(n, H, D, 3, dev)
    cu = prompt.starts(lens, dev)
    want = q.attn_prompt(x, k, v, cu)

    def bounded(limit, stall):
        o, st = torch.full_like(x, float("nan")), status(dev)
        rc = q.qspec_debug_attn_prompt_bounded(x, H * G * D, k, H * D, v, H * D, cu, cu, n, n, B, H * G, H, D, scale, o, H * G * D,
                                               limit, stall, st)
        assert rc == q.OK
        torch.cuda.synchronize()
        return o, read_status(st)

    for _ in range(2):
        assert bounded(SHORT, 1)[1] == q.ERR_TIMEOUT
        o, st = bounded(REGULAR, 0)
        assert st == 0 and torch.equal(o, want)
    if n <= 1100:
        prompt.check(x, k, v, lens, lens, scale, want)
