"""Weights of the FP8 linears quantised on the stream right in front of them: a linear reads its weights ahead of the
dependency on the kernel before it, so the quantiser may let it begin only when they are written."""
import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q, synthetic as syn
from gpuhelp import need_gpu

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("N,K", [(256, 512), (2048, 1024), (4096, 4096)])
def test_quantiser_and_linear_in_a_graph(N, K):
    dev = need_gpu()
    x = syn.activations(5, K, 1, device=dev)
    parents = [(syn.activations(N, K, s, device=dev).float() * 0.02).to(torch.float16) for s in range(2, 6)]
    xq, sa = q.quant_act_fp8(x)
    want = [q.linear_fp8(xq, sa, *q.quant_weights_fp8(p)) for p in parents]
    torch.cuda.synchronize()
    w8, s8 = torch.zeros((N, K), dtype=torch.uint8, device=dev), torch.zeros(N, device=dev)
    out = [torch.empty_like(w) for w in want]
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for p, y in zip(parents, out):                       # (one buffer: the weights of the call before stand in it)
            assert q.qspec_quant_weights_fp8(p, N, K, w8, s8) == 0
            q.linear_fp8(xq, sa, w8, s8, out=y)
    for _ in range(20):
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))


@pytest.mark.parametrize("M", [1, 5, 40, 100, 200])
@pytest.mark.parametrize("N,K", [(256, 512), (2048, 1024), (4096, 4096)])
def test_block_quantiser_and_products_in_a_graph(M, N, K):
    dev = need_gpu()
    parents = [(syn.activations(N, K, s, device=dev).float() * 0.02).to(torch.float16) for s in range(2, 6)]
    xq, sa = q.quant_act_fp8_block(syn.activations(M, K, 1, device=dev))
    up = q.quant_weights_fp8_block(parents[0])
    made = [q.quant_weights_fp8_block(p) for p in parents]
    want = [(q.linear_fp8_block(xq, sa, *w), *q.gated_fp8_block(xq, sa, *w, *up)[:2]) for w in made]
    torch.cuda.synchronize()
    w8, sw = torch.zeros((N, K), dtype=torch.uint8, device=dev), torch.zeros((N // 128, K // 128), device=dev)
    out = []
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        for i, p in enumerate(parents + parents):                # (one buffer: the weights of the call before stand in it)
            assert q.qspec_quant_weights_fp8_block(p, N, K, w8, sw) == 0
            out.append((q.linear_fp8_block(xq, sa, w8, sw),) if i < len(parents) else q.gated_fp8_block(xq, sa, w8, sw, *up)[:2])
    for _ in range(20):
        g.replay()
    torch.cuda.synchronize()
    for i, w in enumerate(want):
        assert torch.equal(out[i][0], w[0]) and torch.equal(out[len(parents) + i][0], w[1]) and torch.equal(out[len(parents) + i][1], w[2])
