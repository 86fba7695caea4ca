"""The two halves of a decoder layer, from library calls only.

Attention (AttentionLayer):
    h = x + residual                                   rmsnorm_fp8 (sum, norm and E4M3 codes in one pass)
    [q k v] = norm(h) W_qkv                            linear_fp8
    cache[b][:, base[b] + i] = 4 bits of (k, v)        kv4_append
    a = attention(q; the cache, or the prompt's rows)  attn_kv4 (draft and verify steps), attn_prompt
    y = a W_out                                        quant_act_fp8, linear_fp8

A prompt's rows attend each other in bf16, as the projection wrote them; the
rows of a later prompt of the same sequences (a prefix in the cache) attend
the cache's entries, read back by kv4_load.  A draft step is one row per
sequence, a verify pass gamma + 1 rows whose entries overwrite the draft's
(both from position `base`).  The class holds no rotary positions and no biases: a
model that has them makes the same calls, with its own step between the projection
and kv4_append.

Feed-forward (FeedForward), E4M3 with a scale for each block of 128:
    h = x + residual                                   rmsnorm_fp8_block
    u = silu(norm(h) W_gate) * (norm(h) W_up)          gated_fp8_block (one kernel, its codes ready for the next call)
    y = u W_down                                       linear_fp8_block

``python -m quantized_speculative_decoding_shared_gb300.layer`` runs prompts, draft
steps and a verify pass through both on seeded inputs.
"""
from __future__ import annotations

import torch

from . import binding as q


class AttentionLayer:
    """Weights, cache and workspace of one layer; w_qkv fp16 [(Hq + 2 H) D][K], w_out fp16 [K][Hq D] (parents of
    the E4M3 weights), w_norm bf16 [K]; B sequences of up to T positions, H KV heads of D.

    Weights, cache and workspace are made on torch's current stream; prompt and step run on `stream` (None: the current
    one), and all that they make belongs to it, their results included.  The cache and the workspace are one to the layer: calls on different
    streams are ordered by the caller, as is a stream's first call after the making."""

    def __init__(self, w_norm, w_qkv, w_out, Hq, H, D, B, T, eps=1e-5):
        dev = w_norm.device
        self.Hq, self.H, self.D, self.B, self.eps = Hq, H, D, B, eps
        self.w_norm = w_norm
        self.status = torch.zeros(1, dtype=torch.int32, device=dev)
        self.w_qkv, self.s_qkv = q.quant_weights_fp8(w_qkv, dev_status=self.status)
        self.w_out, self.s_out = q.quant_weights_fp8(w_out, dev_status=self.status)
        self.cache = q.kv4_cache(B, H, T, D, device=dev)
        self.workspace = q.attn_kv4_workspace(B, 1, Hq, H, D, device=dev)       # any number of rows
        self.each = torch.arange(B + 1, dtype=torch.int32, device=dev)

    def _project(self, x, residual):
        xq, sa, h, _ = q.rmsnorm_fp8(x, self.w_norm, self.eps, residual=residual, dev_status=self.status)
        y = q.linear_fp8(xq, sa, self.w_qkv, self.s_qkv, dev_status=self.status)
        heads = y.view(x.shape[0], self.Hq + 2 * self.H, self.D)
        return h, heads[:, :self.Hq], heads[:, self.Hq:self.Hq + self.H], heads[:, self.Hq + self.H:]

    def _out(self, o):
        xq, sa = q.quant_act_fp8(o.view(o.shape[0], self.Hq * self.D), dev_status=self.status)
        return q.linear_fp8(xq, sa, self.w_out, self.s_out, dev_status=self.status)

    def prompt(self, x, start, base=None, key_start=None, keys=None, residual=None, stream=None):
        """Packed prompt rows x bf16 [rows][K]; start int32 [B + 1].  With a prefix: base int32 [B] positions that the
        cache holds, key_start int32 [B + 1] = cumulated base + rows of each sequence, keys = its last value.
        Returns (y, h): the block's output and the residual stream (None without residual)."""
        if base is not None:
            if key_start is None or not isinstance(keys, int) or keys < 0:
                raise ValueError("a prefix needs key_start and the number of keys")
            if (key_start.device != x.device or key_start.dtype != torch.int32 or key_start.numel() != self.B + 1
                    or not key_start.is_contiguous()):
                raise ValueError("key_start must be contiguous int32 [%d] next to x" % (self.B + 1))
        with q.on_stream(stream):
            if x.shape[0] == 0:                          # (the linears take one row at least)
                return x.new_empty((0, self.w_out.shape[0])), None if residual is None else torch.empty_like(x)
            h, qr, k, v = self._project(x, residual)
            at = torch.zeros_like(self.each[:-1]) if base is None else base
            q.kv4_append(self.cache, k, v, start, at, dev_status=self.status)
            if base is not None:
                k, v = q.kv4_load(self.cache, key_start, torch.zeros_like(at), keys, dev_status=self.status)
            o = q.attn_prompt(qr, k, v, start, key_start if base is not None else None, dev_status=self.status)
            return self._out(o), h

    def step(self, x, base, residual=None, stream=None):
        """R newest rows of every sequence, x bf16 [B R][K], at positions base[b], base[b] + 1, ...: R = 1 drafts,
        R = gamma + 1 verifies.  Returns (y, h)."""
        R, over = divmod(x.shape[0], self.B)
        if over or not 1 <= R <= q.MAX_GAMMA + 1:
            raise ValueError("x must hold 1 to %d rows for each of the %d sequences" % (q.MAX_GAMMA + 1, self.B))
        with q.on_stream(stream):
            h, qr, k, v = self._project(x, residual)
            q.kv4_append(self.cache, k, v, self.each * R, base, dev_status=self.status)
            o = q.attn_kv4(qr, self.cache, base + R, self.D ** -0.5, workspace=self.workspace, dev_status=self.status)
            return self._out(o), h


class FeedForward:
    """Weights of the gated half of a layer: w_gate, w_up fp16 [N][K], w_down fp16 [K][N] (parents of the E4M3 weights),
    w_norm bf16 [K]; N and K multiples of 128.

    The weights are quantised on torch's current stream; run works on `stream` (None: the current one), and all that it
    makes belongs to it, its results included.  It keeps nothing between calls: calls on different streams may overlap, but the
    caller orders a stream's first call after the making.  `status` is one word for the weights and all calls: the first
    error stays in it."""

    def __init__(self, w_norm, w_gate, w_up, w_down, eps=1e-5):
        self.w_norm, self.eps = w_norm, eps
        self.status = torch.zeros(1, dtype=torch.int32, device=w_norm.device)
        self.gate = q.quant_weights_fp8_block(w_gate, dev_status=self.status)
        self.up = q.quant_weights_fp8_block(w_up, dev_status=self.status)
        self.down = q.quant_weights_fp8_block(w_down, dev_status=self.status)

    def run(self, x, residual=None, stream=None):
        """Rows x bf16 [rows][K] of prompts, draft steps or a verify pass.  Returns (y, h): the block's output and the
        residual stream (None without residual)."""
        with q.on_stream(stream):
            if x.shape[0] == 0:                          # (the calls take one row at least)
                return torch.empty_like(x), None if residual is None else torch.empty_like(x)
            xq, sa, h, _ = q.rmsnorm_fp8_block(x, self.w_norm, self.eps, residual=residual, dev_status=self.status)
            hq, sh, _ = q.gated_fp8_block(xq, sa, *self.gate, *self.up, dev_status=self.status)
            return q.linear_fp8_block(hq, sh, *self.down, dev_status=self.status), h


def main():
    from . import synthetic as syn
    dev = torch.device("cuda")
    K, N, Hq, H, D, B, T, gamma = 2048, 5632, 16, 4, 128, 4, 512, 4
    fp16 = lambda n, k, seed: (syn.activations(n, k, seed, device=dev).float() * 0.02).to(torch.float16)   # noqa: E731
    ones = torch.ones(K, dtype=torch.bfloat16, device=dev)
    layer = AttentionLayer(ones, fp16((Hq + 2 * H) * D, K, 1), fp16(K, Hq * D, 2), Hq, H, D, B, T)
    ffn = FeedForward(ones, fp16(N, K, 5), fp16(N, K, 6), fp16(K, N, 7))
    lens = [200, 1, 77, 130]
    start = torch.tensor([0, 200, 201, 278, 408], dtype=torch.int32, device=dev)
    x = syn.activations(sum(lens), K, 3, device=dev)
    y, h = layer.prompt(x, start, residual=syn.activations(sum(lens), K, 4, device=dev))
    y, h = ffn.run(y, residual=h)
    base = torch.tensor(lens, dtype=torch.int32, device=dev)
    for i in range(gamma):
        x = syn.activations(B, K, 10 + i, device=dev)
        y, h = layer.step(x, base + i, residual=x)
        ffn.run(y, residual=h)
    x = syn.activations(B * (gamma + 1), K, 20, device=dev)
    y, h = layer.step(x, base, residual=x)
    y, _ = ffn.run(y, residual=h)
    torch.cuda.synchronize()
    print("prompts of %s rows, %d draft steps, a verify pass of %d rows: status %d, |y| mean %.4f"
          % (lens, gamma, y.shape[0], int((layer.status + ffn.status).item()), float(y.float().abs().mean())))


if __name__ == "__main__":
    main()
