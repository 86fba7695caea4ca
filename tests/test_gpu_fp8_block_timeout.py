"""The bounded waits of the products with block scales, tested without any fault.

Through the diagnostic entry the warp that issues the products waits, with a short bound, on a barrier that nothing
arrives at.  The kernel must give up, walk to its end past every barrier its warps and its cluster share, let its copies
finish, free its tensor memory, report QSPEC_ERR_TIMEOUT and return; a regular call then gives its bits."""
import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q, synthetic as syn
from gpuhelp import need_gpu, read_status, status

pytestmark = pytest.mark.gpu

REGULAR = 1 << 22           # the library's own bound
SHORT = 2000                # a bound the stalled wait runs through


# every width of the few-token kernel, K in parts and whole, fewer blocks than stages and more; tiles in one round, in
# several, all of them in parts, and the last ones in parts
@pytest.mark.parametrize("M,N,K", [(1, 128, 128), (3, 640, 4096), (16, 40960, 512), (30, 256, 2048), (64, 512, 1024), (100, 384, 4096),
                                   (140, 256, 384), (200, 512, 4096), (300, 20480, 256), (130, 39424, 512), (130, 39424, 2048),
                                   (1, 10240, 1536), (7, 6144, 2560), (16, 5120, 2048), (100, 5120, 1280), (50, 4096, 2048)])
@pytest.mark.parametrize("is_gated", [False, True])
def test_then_a_regular_call(M, N, K, is_gated):
    dev = need_gpu()
    xq, sa = q.quant_act_fp8_block(syn.activations(M, K, 1, device=dev))
    w, v = (q.quant_weights_fp8_block((syn.activations(N, K, s, device=dev).float() * 0.05).to(torch.float16)) for s in (2, 3))

    def outputs():
        y = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=dev)
        return y, torch.zeros((M, N), dtype=torch.uint8, device=dev), torch.zeros((N // 128, M), device=dev)

    def bounded(limit, stall):
        (y, hq, sh), st = outputs(), status(dev)
        if is_gated:
            rc = q.qspec_debug_fp8_block_bounded(xq, sa, M, *w, *v, M, N, K, hq, sh, M, y, N, limit, stall, st)
        else:
            rc = q.qspec_debug_fp8_block_bounded(xq, sa, M, *w, None, None, M, N, K, None, None, 0, y, N, limit, stall, st)
        assert rc == q.OK
        torch.cuda.synchronize()                # the kernel returned
        return (y, hq, sh) if is_gated else (y,), read_status(st)

    want = q.gated_fp8_block(xq, sa, *w, *v, want_bf16=True) if is_gated else None
    want = (want[2], want[0], want[1]) if is_gated else (q.linear_fp8_block(xq, sa, *w),)
    for _ in range(2):
        assert bounded(SHORT, 1)[1] == q.ERR_TIMEOUT
        got, st = bounded(REGULAR, 0)
        assert st == 0 and all(torch.equal(a, b) for a, b in zip(got, want))
