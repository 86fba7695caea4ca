"""The layer's own checks: a call that it refuses has not touched the cache (no GPU needed)."""
import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q
from quantized_speculative_decoding_shared_gb300.layer import AttentionLayer

B, K, Hq, H, D = 3, 256, 4, 2, 64


@pytest.fixture
def layer(monkeypatch):
    """A layer of three sequences whose library calls are counted instead of made."""
    made = []

    def stub(name, *widths):
        def call(t, *args, **kw):
            made.append(name)
            n = t[0].shape[0] if isinstance(t, tuple) else t.shape[0]
            out = tuple(torch.zeros((n, w), dtype=torch.bfloat16) for w in widths)
            return out if len(out) > 1 else out[0]
        monkeypatch.setattr(q, name, call)

    stub("rmsnorm_fp8", K, 1, K, K)
    stub("linear_fp8", (Hq + 2 * H) * D)
    stub("quant_act_fp8", Hq * D, 1)
    for name in ("attn_prompt", "attn_kv4"):
        stub(name, Hq * D)
    for name in ("kv4_append", "kv4_load"):
        monkeypatch.setattr(q, name, lambda *args, name=name, **kw: made.append(name) or (x(0), x(0)))
    layer = AttentionLayer.__new__(AttentionLayer)
    layer.B, layer.Hq, layer.H, layer.D, layer.eps = B, Hq, H, D, 1e-5
    layer.w_norm = layer.w_qkv = layer.s_qkv = layer.s_out = layer.cache = layer.workspace = layer.status = None
    layer.w_out = torch.zeros((K, Hq * D), dtype=torch.uint8)
    layer.each = torch.arange(B + 1, dtype=torch.int32)
    return layer, made


def x(rows):
    return torch.zeros((rows, K), dtype=torch.bfloat16)


@pytest.mark.parametrize("rows", [0, 1, 7, 3 * 18])
def test_step_refuses_before_it_writes(layer, rows):
    """Rows that are no whole number of rows to a sequence, none, or more than a verify pass has."""
    layer, made = layer
    with pytest.raises(ValueError):
        layer.step(x(rows), torch.zeros(B, dtype=torch.int32))
    assert "kv4_append" not in made


@pytest.mark.parametrize("change", [dict(key_start=None), dict(keys=None), dict(keys=-1), dict(keys=2.5),
                                    dict(key_start=torch.zeros(B, dtype=torch.int32)),
                                    dict(key_start=torch.zeros(B + 1, dtype=torch.int64))])
def test_prompt_with_a_prefix_refuses_before_it_writes(layer, change):
    layer, made = layer
    starts = torch.zeros(B + 1, dtype=torch.int32)
    prefix = dict(base=torch.zeros(B, dtype=torch.int32), key_start=starts, keys=6)
    with pytest.raises(ValueError):
        layer.prompt(x(6), starts, **dict(prefix, **change))
    assert "kv4_append" not in made


@pytest.mark.parametrize("residual", [False, True])
def test_a_prompt_without_rows(layer, residual):
    """A step in which every sequence is empty: no rows out, and nothing called."""
    layer, made = layer
    starts = torch.zeros(B + 1, dtype=torch.int32)
    for prefix in ({}, dict(base=torch.ones(B, dtype=torch.int32), key_start=starts, keys=3)):
        y, h = layer.prompt(x(0), starts, residual=x(0) if residual else None, **prefix)
        assert y.shape == (0, K) and y.dtype == torch.bfloat16 and made == []
        assert h.shape == (0, K) if residual else h is None
