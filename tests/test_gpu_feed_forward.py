"""The feed-forward half of a layer (layer.py): every call's result against its definition on what the call before it
gave, alone and behind the attention half; in a captured graph, on other streams, and several at once."""
import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q, synthetic as syn
from quantized_speculative_decoding_shared_gb300.layer import AttentionLayer, FeedForward
from blockref import act_values, check_codes, check_linear, gated, weight_codes, weight_values
from gpuhelp import need_gpu, read_status, status

pytestmark = pytest.mark.gpu
K, N, EPS = 512, 1152, 1e-5


def fp16(n, k, seed, dev):
    return (syn.activations(n, k, seed, device=dev).float() * 0.05).to(torch.float16)


def norm_weights(dev):
    return (1 + 0.1 * syn.activations(1, K, 5, device=dev).float()).to(torch.bfloat16).view(K)


def block(dev, seed=1):
    return FeedForward(norm_weights(dev), fp16(N, K, seed, dev), fp16(N, K, seed + 1, dev), fp16(K, N, seed + 2, dev), EPS)


class Recorder:
    def __init__(self, monkeypatch):
        self.calls = {}
        for name in ("rmsnorm_fp8_block", "gated_fp8_block", "linear_fp8_block"):
            monkeypatch.setattr(q, name, self.wrap(name, getattr(q, name)))

    def wrap(self, name, f):
        def call(*args, **kw):
            assert name not in self.calls
            r = f(*args, **kw)
            self.calls[name] = r
            return r
        return call


def check(ffn, rec, x, r, y, h):
    xq, sa, hh, _ = rec.calls["rmsnorm_fp8_block"]
    a = x.float() if r is None else (x.float() + r.float()).to(torch.bfloat16).float()
    assert h is None if r is None else torch.equal(h.float(), a)
    ref = a.double() / torch.sqrt((a.double() ** 2).mean(-1, keepdim=True) + EPS) * ffn.w_norm.double()
    check_codes(xq, sa, ref, ref.abs() * 64 * 2.0 ** -24)                # (the norm's own bound)
    hq, sh, _ = rec.calls["gated_fp8_block"]
    check_codes(hq, sh, *gated(act_values(xq, sa), weight_values(*ffn.gate), weight_values(*ffn.up)))
    assert y is rec.calls["linear_fp8_block"]
    check_linear(y, act_values(hq, sh), weight_values(*ffn.down))
    rec.calls.clear()


@pytest.mark.parametrize("rows", [1, 3, 20, 65, 200])
@pytest.mark.parametrize("residual", [False, True])
def test_every_call(rows, residual, monkeypatch):
    dev = need_gpu()
    ffn, rec = block(dev), Recorder(monkeypatch)
    for w, parent in zip((ffn.gate, ffn.up, ffn.down), (fp16(N, K, 1, dev), fp16(N, K, 2, dev), fp16(K, N, 3, dev))):
        want = weight_codes(parent)
        assert torch.equal(w[0].cpu(), want[0]) and torch.equal(w[1].cpu(), want[1])
    x = syn.activations(rows, K, 7, device=dev, outlier_frac=0.01)
    r = syn.activations(rows, K, 8, device=dev) if residual else None
    y, h = ffn.run(x, residual=r)
    check(ffn, rec, x, r, y, h)
    assert read_status(ffn.status) == 0


def test_behind_the_attention(monkeypatch):
    """Prompts, a draft step and a verify pass through both halves."""
    dev = need_gpu()
    B, T, gamma, Hq, H, D, lens = 3, 300, 3, 8, 2, 64, [150, 1, 37]
    att = AttentionLayer(norm_weights(dev), fp16((Hq + 2 * H) * D, K, 1, dev), fp16(K, Hq * D, 2, dev), Hq, H, D, B, T, EPS)
    ffn, rec = block(dev, 11), Recorder(monkeypatch)
    start, base = (torch.tensor(v, dtype=torch.int32, device=dev) for v in ([0, 150, 151, 188], lens))
    x = syn.activations(sum(lens), K, 3, device=dev)
    for y, h in (att.prompt(x, start, residual=x), att.step(x[:B], base, residual=x[:B]),
                 att.step(x[:B * (gamma + 1)], base, residual=x[:B * (gamma + 1)])):
        out, hh = ffn.run(y, residual=h)
        check(ffn, rec, y, h, out, hh)
    assert read_status(att.status) == 0 and read_status(ffn.status) == 0


def test_no_rows():
    dev = need_gpu()
    ffn = block(dev)
    x = torch.empty((0, K), dtype=torch.bfloat16, device=dev)
    y, h = ffn.run(x)
    assert y.shape == (0, K) and y.dtype == torch.bfloat16 and h is None
    y, h = ffn.run(x, residual=x)
    assert y.shape == (0, K) and h.shape == (0, K)


def test_in_a_graph_with_weights_made_in_front():
    """Weights quantised, used and made anew within one captured graph: the products read theirs, not those of the last
    replay, however closely the launches follow one another."""
    dev = need_gpu()
    rows = [1, 17, 70, 300]
    xs = [syn.activations(m, K, 20 + m, device=dev) for m in rows]
    parents = [fp16(n, k, 30, dev) for n, k in ((N, K), (N, K), (K, N))]

    def program():
        out = []
        for i, x in enumerate(xs):
            scale = 1.0 + i
            gate, up, down = (q.quant_weights_fp8_block((p.float() * scale).to(torch.float16)) for p in parents)
            out.append(q.linear_fp8_block(*q.gated_fp8_block(*q.quant_act_fp8_block(x), *gate, *up)[:2], *down))
            hq = q.quant_act_fp8_block(wide[i])
            out.append(q.linear_fp8_block(*hq, *q.quant_weights_fp8_block(parents[2])))     # the weights, then at once the product
        return out

    wide = [syn.activations(m, N, 40 + m, device=dev) for m in rows]
    want = [t.clone() for t in program()]
    torch.cuda.synchronize()
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = program()
    for _ in range(3):
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert [i for i, (a, b) in enumerate(zip(got, want)) if not torch.equal(a, b)] == []
        held = [p.clone() for p in parents]                 # other weights: the results change, and change back
        for p in parents:
            p.mul_(0.5)
        g.replay()
        torch.cuda.synchronize()
        assert not any(torch.equal(a, b) for a, b in zip(got, want))
        for p, t in zip(parents, held):
            p.copy_(t)


@pytest.mark.parametrize("kind", ["object", "handle"])
def test_on_a_given_stream(kind):
    """Results belong to the given stream, the current one being busy meanwhile."""
    dev = need_gpu()
    ffn = block(dev)
    x = syn.activations(40, K, 3, device=dev)
    want = ffn.run(x, residual=x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda._sleep(20_000_000)
    got = ffn.run(x, residual=x, stream=s if kind == "object" else s.cuda_stream)
    junk = [torch.full((40, K), 7.0, dtype=torch.bfloat16, device=dev) for _ in range(8)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want)) and len(junk) == 8


def test_two_streams_at_once():
    """Calls that overlap on the GPU, split over clusters and not, give what they give alone."""
    dev = need_gpu()
    cases = []
    for i, (m, n, k) in enumerate([(1, 1024, 4096), (70, 256, 2048), (200, 1280, 1024), (30, 512, 512)]):
        xq, sa = q.quant_act_fp8_block(syn.activations(m, k, i, device=dev))
        w, v = (q.quant_weights_fp8_block(fp16(n, k, 10 * i + j, dev)) for j in (1, 2))
        cases.append((xq, sa, w, v))
    run = lambda c, st=None, stream=None: (q.linear_fp8_block(c[0], c[1], *c[2], dev_status=st, stream=stream),   # noqa: E731
                                           *q.gated_fp8_block(c[0], c[1], *c[2], *c[3], dev_status=st, stream=stream)[:2])
    want = [run(c) for c in cases]
    torch.cuda.synchronize()
    streams, st, got = [torch.cuda.Stream() for _ in range(3)], status(dev), []
    for rep in range(20):
        for j, s in enumerate(streams):
            c = (rep + j) % len(cases)
            got.append((c, run(cases[c], st, s)))
    torch.cuda.synchronize()
    assert read_status(st) == 0
    for c, r in got:
        assert all(torch.equal(a, b) for a, b in zip(r, want[c]))


def test_the_same_bits_every_time():
    """Parts of K meet in a fixed order."""
    dev = need_gpu()
    for m, n, k in [(3, 512, 8192), (100, 256, 4096), (150, 768, 3584), (300, 256, 8192)]:
        xq, sa = q.quant_act_fp8_block(syn.activations(m, k, 1, device=dev))
        w, v = (q.quant_weights_fp8_block(fp16(n, k, j, dev)) for j in (1, 2))
        y, h = q.linear_fp8_block(xq, sa, *w), q.gated_fp8_block(xq, sa, *w, *v)[:2]
        for _ in range(10):
            assert torch.equal(q.linear_fp8_block(xq, sa, *w), y)
            assert all(torch.equal(a, b) for a, b in zip(q.gated_fp8_block(xq, sa, *w, *v)[:2], h))
