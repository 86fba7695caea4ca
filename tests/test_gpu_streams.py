"""Calls on a stream that is not torch's current one, given as a stream object or as a raw handle.

The current stream is kept busy meanwhile, so that a fill or an allocation of the call's own that went to it instead
of the given stream would come after the kernel and show in the result."""
import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q, synthetic as syn
from quantized_speculative_decoding_shared_gb300.layer import AttentionLayer
from gpuhelp import need_gpu, read_status, status
from layerref import random_cache

pytestmark = pytest.mark.gpu
BUSY = 20_000_000                               # clocks that the current stream is kept busy for: some 10 ms


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def given(kind):
    """A stream other than the current one, and what a call is given for it."""
    s = torch.cuda.Stream()
    return s, (s if kind == "object" else s.cuda_stream)


def on_a_busy_device(call):
    """The call's results, as they are once everything queued is done; the current stream is busy during the call."""
    torch.cuda.synchronize()
    torch.cuda._sleep(BUSY)
    got = call()
    torch.cuda.synchronize()
    return got


@pytest.mark.parametrize("kind", ["object", "handle"])
def test_rows_read_back(kind):
    dev = need_gpu()
    cache = random_cache(2, 4, 64, 128, 3, dev)
    start, base = ints([0, 40, 70], dev), ints([5, 30], dev)
    want = q.kv4_load(cache, start, base, 70)
    s, arg = given(kind)
    got = on_a_busy_device(lambda: q.kv4_load(cache, start, base, 70, stream=arg))
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.any(want[0] != 0)


@pytest.mark.parametrize("kind", ["object", "handle"])
def test_cache_attention_with_a_workspace_of_its_own(kind):
    """The workspace's counters are zeros when the kernel begins: the memory it comes from holds something else, and
    several CTAs have parts of each task."""
    dev = need_gpu()
    B, R, H, G, D, T = 2, 3, 4, 2, 128, 3000
    cache = random_cache(B, H, T, D, 4, dev)
    x = syn.activations(B * R * H * G, D, 5, device=dev).view(B * R, H * G, D)
    length = ints([3000, 2500], dev)
    want = q.attn_kv4(x, cache, length, 0.1)
    n = q.qspec_attn_kv4_workspace_bytes(B, R, H * G, H, D)
    s, arg = given(kind)
    with torch.cuda.stream(s):                          # (a block of the given stream's pool, and one of the current's)
        torch.full((n,), 1, dtype=torch.uint8, device=dev)
    torch.full((n,), 1, dtype=torch.uint8, device=dev)
    st = status(dev)
    got = on_a_busy_device(lambda: q.attn_kv4(x, cache, length, 0.1, dev_status=st, stream=arg))
    assert read_status(st) == 0 and torch.equal(got, want)


@pytest.mark.parametrize("kind", ["object", "handle"])
def test_prompts_drafts_and_verify_of_a_layer(kind):
    """A layer's program on a given stream, and what the current stream's allocations do meanwhile, leave the same bits
    as the program on the current stream."""
    dev = need_gpu()
    B, T, gamma, K, Hq, H, D, lens = 3, 300, 3, 512, 8, 2, 128, [150, 1, 37]
    w = torch.ones(K, dtype=torch.bfloat16, device=dev)
    fp16 = lambda n, k, seed: (syn.activations(n, k, seed, device=dev).float() * 0.05).to(torch.float16)   # noqa: E731
    layer = AttentionLayer(w, fp16((Hq + 2 * H) * D, K, 1), fp16(K, Hq * D, 2), Hq, H, D, B, T)
    x, res = syn.activations(sum(lens), K, 3, device=dev), syn.activations(sum(lens), K, 4, device=dev)
    start, at = ints([0, 150, 151, 188], dev), [ints([n + i for n in lens], dev) for i in range(gamma)]
    held = ints([n + gamma + 1 for n in lens], dev)
    more, start2, total = syn.activations(25, K, 30, device=dev), ints([0, 5, 5, 25], dev), [lens[0] + 9, lens[1] + 4, lens[2] + 24]
    key_start, keys = ints([0, total[0], total[0] + total[1], sum(total)], dev), sum(total)
    drafts = [syn.activations(B, K, 10 + i, device=dev) for i in range(gamma)]
    rows = syn.activations(B * (gamma + 1), K, 20, device=dev)

    def program(between=lambda: None, **kw):
        out = list(layer.prompt(x, start, residual=res, **kw))
        for d, p in zip(drafts, at):
            between()
            out.append(layer.step(d, p, **kw)[0])
        between()
        out.append(layer.step(rows, at[0], **kw)[0])
        between()
        out.append(layer.prompt(more, start2, base=held, key_start=key_start, keys=keys, **kw)[0])
        between()
        return out

    want = program()
    cache = [t.clone() for t in layer.cache]
    s, arg = given(kind)
    for late in (False, True):                              # the current stream late, the given one late
        for t in layer.cache:
            t.zero_()

        def others():                                       # the current stream's memory, used again at once
            for n in (16, 1024, 1 << 16, 1 << 18, 1 << 20):
                torch.full((n,), 0xFF, dtype=torch.uint8, device=dev)

        torch.cuda.synchronize()
        if late:
            with torch.cuda.stream(s):
                torch.cuda._sleep(BUSY)
        else:
            torch.cuda._sleep(BUSY)
        got = program(others, stream=arg)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a, b) for a, b in zip(layer.cache, cache))
    assert read_status(layer.status) == 0


def calls(dev):
    """The calls that make their outputs, on inputs of a few rows."""
    M, N, K, V = 5, 256, 512, 1000
    x, w = syn.activations(M, K, 1, device=dev), torch.ones(K, dtype=torch.bfloat16, device=dev)
    codes, sc, z = syn.weights(N, K, 2, device=dev)
    packed, sz = q.pack_weights(codes, sc, z)
    w16 = (syn.activations(N, K, 3, device=dev).float() * 0.05).to(torch.float16)
    w8, s8 = q.quant_weights_fp8(w16)
    x4, x8 = q.quant_act_int4(x), q.quant_act_fp8(x)
    p = syn.activations(2 * 4, V, 4, device=dev).view(2, 4, V)
    p3, p0, none, lens = p[:, :3].contiguous(), p[:, 0].contiguous(), ints([0, 0], dev), ints([70, 50], dev)
    draft = ints([[1, 2, 3], [4, 5, 6]], dev)
    h = syn.activations(70 * 8, 64, 6, device=dev).view(70, 8, 64)
    cu = ints([0, 30, 70], dev)
    cache = random_cache(2, 2, 70, 64, 3, dev)
    return {
        "pack_weights": lambda **kw: q.pack_weights(codes, sc, z, **kw),
        "quant_act_int4": lambda **kw: q.quant_act_int4(x, **kw),
        "linear_w4a4": lambda **kw: q.linear_w4a4(*x4, packed, sz, **kw),
        "linear_w4a4_bf16": lambda **kw: q.linear_w4a4_bf16(x, packed, sz, **kw),
        "linear_w4a16": lambda **kw: q.linear_w4a16(x, packed, sz, **kw),
        "verify_greedy": lambda **kw: q.verify_greedy(p, draft, **kw),
        "verify_sample": lambda **kw: q.verify_sample(p, p3, draft, 7, 1, **kw),
        "draft_sample": lambda **kw: q.draft_sample(p0, 7, 1, 1, **kw),
        "quant_weights_fp8": lambda **kw: q.quant_weights_fp8(w16, **kw),
        "quant_act_fp8": lambda **kw: q.quant_act_fp8(x, **kw),
        "linear_fp8": lambda **kw: q.linear_fp8(*x8, w8, s8, **kw),
        "rmsnorm_fp8": lambda **kw: q.rmsnorm_fp8(x, w, 1e-5, residual=x, want_bf16=True, **kw),
        "kv4_load": lambda **kw: q.kv4_load(cache, cu, none, 70, **kw),
        "attn_kv4": lambda **kw: q.attn_kv4(h[:6], cache, lens, 0.1, **kw),
        "attn_prompt": lambda **kw: q.attn_prompt(h, h[:, :2], h[:, 2:4], cu, **kw),
    }


@pytest.mark.parametrize("name", ["pack_weights", "quant_act_int4", "linear_w4a4", "linear_w4a4_bf16", "linear_w4a16", "verify_greedy",
                                  "verify_sample", "draft_sample", "quant_weights_fp8", "quant_act_fp8", "linear_fp8", "rmsnorm_fp8",
                                  "kv4_load", "attn_kv4", "attn_prompt"])
@pytest.mark.parametrize("kind", ["object", "handle"])
def test_outputs_are_memory_of_the_given_stream(name, kind):
    """Memory that the current stream still writes (dropped by the program, its last fill queued) is not what a call on
    another stream puts its results into."""
    dev = need_gpu()
    call = calls(dev)[name]
    tensors = lambda r: list(r) if isinstance(r, tuple) else [r]            # noqa: E731
    want = [t.clone() for t in tensors(call())]
    s, arg = given(kind)

    def fill():
        for t in [torch.empty_like(t) for t in want]:
            t.view(torch.uint8).fill_(0x11)

    def fills_then_call():
        fill()
        return tensors(call(stream=arg))

    got = on_a_busy_device(fills_then_call)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


@pytest.mark.parametrize("kind", ["zero", "legacy", "per thread", "default", "external"])
def test_other_ways_to_name_a_stream(kind):
    """The default stream by its handles and as an object, a thread's own stream, a handle wrapped as a stream."""
    dev = need_gpu()
    own = torch.cuda.Stream()
    arg = {"zero": 0, "legacy": 1, "per thread": 2, "default": torch.cuda.default_stream(),
           "external": torch.cuda.ExternalStream(own.cuda_stream)}[kind]
    call = calls(dev)
    for name in ("rmsnorm_fp8", "kv4_load", "attn_kv4"):
        want = call[name]()
        torch.cuda.synchronize()
        got = call[name](stream=arg)
        torch.cuda.synchronize()
        for a, b in zip(*(t if isinstance(t, tuple) else (t,) for t in (got, want))):
            assert torch.equal(a, b), name
