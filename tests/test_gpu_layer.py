"""The attention half of a decoder layer (layer.py): every call's result against the definition, on what the call
before it gave, so that each tolerance is the call's own.

Cache entries: bit-exact.  Attention: (2^-8 + 2^-12 + 2 d) A + 2^-8 |o| with A = sum p |v| and d the error of a score
(16 x 2^-24 of its largest sum of magnitudes).  Linears: 1e-2 (1 + |ref|), their own bound."""
import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q, synthetic as syn
from quantized_speculative_decoding_shared_gb300.layer import AttentionLayer
from gpuhelp import need_gpu, read_status
from layerref import attention, pack, quantise_rows, values, words

pytestmark = pytest.mark.gpu
K, EPS = 512, 1e-5


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def starts(lens, dev):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return ints(at, dev)


class Recorder:
    """The library's calls of a layer, each with its arguments and result."""

    def __init__(self, monkeypatch):
        self.calls = []
        for name in ("rmsnorm_fp8", "linear_fp8", "kv4_append", "kv4_load", "attn_prompt", "attn_kv4", "quant_act_fp8"):
            monkeypatch.setattr(q, name, self.wrap(name, getattr(q, name)))

    def wrap(self, name, f):
        def call(*args, **kw):
            r = f(*args, **kw)
            self.calls.append((name, args, r))
            return r
        return call

    def take(self, *names):
        assert [c[0] for c in self.calls] == list(names)
        got, self.calls = self.calls, []
        return got


def check_linear(call):
    xq, sa, w8, s8 = call[1][:4]
    ref = ((xq.view(torch.float8_e4m3fn).double() @ w8.view(torch.float8_e4m3fn).double().T) * sa.double()[:, None]
           * s8.double())
    assert torch.all((call[2].double() - ref).abs() <= 1e-2 * (1 + ref.abs()))


def check_head(x, k, v, first, scale, o, top):
    ref, A = attention(x, k, v, first, scale)
    d = 16 * 2.0 ** -24 * scale * top
    assert torch.all((o - ref).abs() <= (2.0 ** -8 + 2.0 ** -12 + 2 * d) * A + 2.0 ** -8 * ref.abs() + 1e-30)


@pytest.mark.parametrize("Hq,H,D", [(8, 2, 128), (6, 2, 64)])
def test_prompt_drafts_and_verify(Hq, H, D, monkeypatch):
    dev = need_gpu()
    B, T, gamma, lens = 3, 400, 3, [150, 1, 37]
    fp16 = lambda n, k, seed: (syn.activations(n, k, seed, device=dev).float() * 0.05).to(torch.float16)   # noqa: E731
    w = (1 + 0.1 * syn.activations(1, K, 5, device=dev).float()).to(torch.bfloat16).view(K)
    layer = AttentionLayer(w, fp16((Hq + 2 * H) * D, K, 1), fp16(K, Hq * D, 2), Hq, H, D, B, T, EPS)
    want = [t.clone() for t in layer.cache]
    rec, scale = Recorder(monkeypatch), D ** -0.5

    def check_append(call, counts, base):
        k, v = call[1][1], call[1][2]
        at = 0
        for b, (n, p) in enumerate(zip(counts, base)):
            for x, codes, sz in ((k, want[0], want[1]), (v, want[2], want[3])):
                c, s, z = quantise_rows(x[at:at + n])
                codes[b, :, p:p + n] = pack(c).transpose(0, 1)
                sz[b, :, p:p + n] = words(s, z).transpose(0, 1)
            at += n
        assert all(torch.equal(a, b) for a, b in zip(layer.cache, want))

    def check_norm(call, x, r):
        xq, sa, h, _ = call[2]
        hh = x if r is None else (x.float() + r.float()).to(torch.bfloat16)
        assert h is None if r is None else torch.equal(h, hh)
        a = hh.double()
        ref = a / torch.sqrt((a * a).mean(-1, keepdim=True) + EPS) * w.double()
        code = xq.view(torch.float8_e4m3fn).double() * sa.double()[:, None]
        step = ref.abs().amax(-1, keepdim=True) / 448
        assert torch.all((code - ref).abs() <= ref.abs() * (2.0 ** -4 + 2.0 ** -18) + step * 2.0 ** -10)

    def seen(b, h, n):
        return (values(want[0][b, h, :n], want[1][b, h, :n]), values(want[2][b, h, :n], want[3][b, h, :n]))

    def check_attn(call, R, length):
        x, o = call[1][0].double(), call[2].double()
        for b, n in enumerate(length):
            for j in range(Hq):
                k, v = seen(b, j // (Hq // H), n)
                s = (want[1][b, j // (Hq // H), :n] & 0xFFFF).to(torch.int16).view(torch.float16).double()
                xx = x[b * R:b * R + R, j]
                check_head(xx, k, v, n - R, scale, o[b * R:b * R + R, j], float(s.max()) * 143 * xx.abs().sum(-1, keepdim=True))

    # prompts, in bf16
    x, r = syn.activations(sum(lens), K, 3, device=dev), syn.activations(sum(lens), K, 4, device=dev)
    layer.prompt(x, starts(lens, dev), residual=r)
    norm, qkv, app, att, _, out = rec.take("rmsnorm_fp8", "linear_fp8", "kv4_append", "attn_prompt", "quant_act_fp8", "linear_fp8")
    check_norm(norm, x, r)
    check_linear(qkv)
    check_append(app, lens, [0] * B)
    check_linear(out)
    at = 0
    for n in lens:
        for j in range(Hq):
            xx, k, v = (t[at:at + n, i].double() for t, i in ((att[1][0], j), (att[1][1], j // (Hq // H)), (att[1][2], j // (Hq // H))))
            check_head(xx, k, v, 0, scale, att[2][at:at + n, j].double(), (xx.abs() @ k.abs().T).amax(-1, keepdim=True))
        at += n
    # draft steps, then the verify pass over their places
    base = ints(lens, dev)
    for i in range(gamma):
        x = syn.activations(B, K, 10 + i, device=dev)
        layer.step(x, base + i)
        norm, qkv, app, att, _, out = rec.take("rmsnorm_fp8", "linear_fp8", "kv4_append", "attn_kv4", "quant_act_fp8", "linear_fp8")
        check_norm(norm, x, None)
        check_append(app, [1] * B, [n + i for n in lens])
        check_attn(att, 1, [n + i + 1 for n in lens])
        check_linear(out)
    x = syn.activations(B * (gamma + 1), K, 20, device=dev)
    layer.step(x, base)
    norm, qkv, app, att, _, out = rec.take("rmsnorm_fp8", "linear_fp8", "kv4_append", "attn_kv4", "quant_act_fp8", "linear_fp8")
    check_append(app, [gamma + 1] * B, lens)
    check_attn(att, gamma + 1, [n + gamma + 1 for n in lens])
    check_linear(out)
    # a second prompt behind what the cache holds
    held, more = [n + gamma + 1 for n in lens], [5, 140, 0]
    total = [a + b for a, b in zip(held, more)]
    x = syn.activations(sum(more), K, 30, device=dev)
    layer.prompt(x, starts(more, dev), base=ints(held, dev), key_start=starts(total, dev), keys=sum(total))
    norm, qkv, app, load, att, _, out = rec.take("rmsnorm_fp8", "linear_fp8", "kv4_append", "kv4_load", "attn_prompt", "quant_act_fp8",
                                                 "linear_fp8")
    check_append(app, more, held)
    k, v = load[2]
    at, kt = 0, 0
    for b, (n, m) in enumerate(zip(more, total)):
        for h in range(H):
            kk, vv = seen(b, h, m)
            assert torch.equal(k[kt:kt + m, h], kk.to(torch.bfloat16)) and torch.equal(v[kt:kt + m, h], vv.to(torch.bfloat16))
        for j in range(Hq):
            xx, kk, vv = att[1][0][at:at + n, j].double(), k[kt:kt + m, j // (Hq // H)].double(), v[kt:kt + m, j // (Hq // H)].double()
            if n:
                check_head(xx, kk, vv, m - n, scale, att[2][at:at + n, j].double(), (xx.abs() @ kk.abs().T).amax(-1, keepdim=True))
        at, kt = at + n, kt + m
    assert read_status(layer.status) == 0


def test_command(capsys):
    need_gpu()
    from quantized_speculative_decoding_shared_gb300 import layer
    layer.main()
    assert "status 0" in capsys.readouterr().out


def test_steps_and_prompts_in_a_graph():
    """Draft steps, a verify pass and a prompt captured on a stream of their own give what the calls give."""
    dev = need_gpu()
    B, T, gamma, Hq, H, D = 2, 300, 2, 8, 2, 128
    fp16 = lambda n, k, seed: (syn.activations(n, k, seed, device=dev).float() * 0.05).to(torch.float16)   # noqa: E731
    layer = AttentionLayer(torch.ones(K, dtype=torch.bfloat16, device=dev), fp16((Hq + 2 * H) * D, K, 1), fp16(K, Hq * D, 2), Hq, H, D,
                           B, T, EPS)
    lens = [120, 33]
    prompt, base, start = syn.activations(sum(lens), K, 3, device=dev), ints(lens, dev), starts(lens, dev)
    res = syn.activations(sum(lens), K, 4, device=dev)
    drafts = [syn.activations(B, K, 10 + i, device=dev) for i in range(gamma)]
    rows = syn.activations(B * (gamma + 1), K, 20, device=dev)

    def program():
        out = list(layer.prompt(prompt, start, residual=res))
        for i, x in enumerate(drafts):
            out.append(layer.step(x, base + i)[0])
        return out + [layer.step(rows, base)[0]]

    want = [t.clone() for t in program()]
    cache = [t.clone() for t in layer.cache]
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = program()
    for _ in range(3):
        for t in layer.cache:
            t.zero_()
        for t in got:
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        for a, b in zip(layer.cache, cache):                           # (the positions in use)
            for i, n in enumerate(lens):
                assert torch.equal(a[i, :, :n + gamma + 1], b[i, :, :n + gamma + 1])
    assert read_status(layer.status) == 0
