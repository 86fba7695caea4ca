"""Causal attention of packed prompts (qspec_attn_prompt) against the formula in 64 bits.

Tolerance of an output o = sum p v, with A = sum p |v|: the weights are rounded
to bf16 (half a step, 2^-8), the exponential is within 2^-12, a score within
d = 16 x 2^-24 x scale max_j sum |q| |k_j| (fp32 sums of exact products), which
counts twice (weight and sum): together (2^-8 + 2^-12 + 2 d) A; and the output is
rounded to bf16: 2^-8 |o|."""
import math

import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q, synthetic as syn
from gpuhelp import need_gpu, read_status, status
from layerref import attention

pytestmark = pytest.mark.gpu


def heads(rows, H, D, seed, dev):
    return syn.activations(max(1, rows * H), D, seed, device=dev, outlier_frac=0.02)[:rows * H].view(rows, H, D)


def starts(lens, dev):
    at = [0]
    for n in lens:
        at.append(at[-1] + n)
    return torch.tensor(at, dtype=torch.int32, device=dev)


def check(x, k, v, lq, lk, scale, o, rows=None):
    G = x.shape[1] // k.shape[1]
    a = c = 0
    for n, m in zip(lq, lk):
        for j in range(x.shape[1]):
            if n == 0:
                continue
            qq, kk, vv = x[a:a + n, j].double(), k[c:c + m, j // G].double(), v[c:c + m, j // G].double()
            first = m - n
            if rows is not None:                       # some rows of a long sequence
                at = torch.tensor([r for r in rows if r < n], device=x.device)
            else:
                at = torch.arange(n, device=x.device)
            got = o[a:a + n, j][at].double()
            if rows is None:
                ref, A = attention(qq, kk, vv, first, scale)
            else:
                parts = [attention(qq[i:i + 1], kk, vv, first + i, scale) for i in at.tolist()]
                ref, A = torch.cat([p[0] for p in parts]), torch.cat([p[1] for p in parts])
            fin = torch.where(torch.isfinite(kk), kk, torch.zeros_like(kk))
            top = (qq[at].abs() @ fin.abs().T).amax(-1, keepdim=True) if m else torch.zeros((len(at), 1), device=x.device)
            d = 16 * 2.0 ** -24 * abs(scale) * top
            tol = (2.0 ** -8 + 2.0 ** -12 + 2 * d) * A + 2.0 ** -8 * ref.abs() + 1e-30
            err = (got - ref).abs()
            assert torch.all(err <= tol), (n, m, j, float((err - tol).max()), float((err / tol).max()))
        a, c = a + n, c + m


def run(lq, lk, H, G, D, seed, scale=None):
    dev = need_gpu()
    scale = 1 / math.sqrt(D) if scale is None else scale
    x, k, v = heads(sum(lq), H * G, D, seed, dev), heads(sum(lk), H, D, seed + 1, dev), heads(sum(lk), H, D, seed + 2, dev)
    st = status(dev)
    o = q.attn_prompt(x, k, v, starts(lq, dev), starts(lk, dev), scale, dev_status=st)
    assert read_status(st) == 0
    check(x, k, v, lq, lk, scale, o)
    return x, k, v, o


@pytest.mark.parametrize("H,G", [(1, 1), (2, 4), (1, 7), (3, 2)])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens", [[1], [2, 0, 31, 64], [127, 128, 129], [255, 1, 257], [513], [0, 0, 5]])
def test_packed_lengths(H, G, D, lens):
    run(lens, lens, H, G, D, 1)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lq,lk", [([1, 1, 1], [500, 1, 129]), ([40, 128, 7], [300, 128, 135]), ([130], [1000]),
                                   ([300, 200], [100, 0]), ([260, 5], [256, 300]), ([64], [63])])
def test_prefixes_and_rows_that_see_nothing(D, lq, lk):
    """Lk > Lq: a prefix; Lk < Lq: the first rows see nothing and are 0."""
    x, k, v, o = run(lq, lk, 2, 2, D, 5)
    a = 0
    for n, m in zip(lq, lk):
        if m < n:
            assert torch.all(o[a:a + n - m] == 0)
        a += n


@pytest.mark.parametrize("scale", [0.0, 2.0, -0.3])
def test_scales(scale):
    run([200, 77], [200, 77], 2, 2, 128, 9, scale)


@pytest.mark.parametrize("D", [64, 128])
def test_growing_scores(D):
    """Keys whose scores rise along the sequence by far more than any rescaling threshold, and fall again."""
    dev = need_gpu()
    n = 700
    x, k, v = heads(n, 2, D, 1, dev), heads(n, 1, D, 2, dev), heads(n, 1, D, 3, dev)
    ramp = torch.cat((torch.linspace(0, 60, 400, device=dev), torch.linspace(60, 1, 300, device=dev)))
    x = (x.float() * 0.1 + 1.0).to(torch.bfloat16)
    k = (k.float() * 0.1 + ramp[:, None, None] / 8).to(torch.bfloat16)
    st = status(dev)
    o = q.attn_prompt(x, k, v, starts([n], dev), dev_status=st)
    assert read_status(st) == 0
    check(x, k, v, [n], [n], 1 / math.sqrt(D), o)


def test_long_sequence_on_some_rows():
    dev = need_gpu()
    n = 4100
    x, k, v = heads(n, 4, 128, 1, dev), heads(n, 2, 128, 2, dev), heads(n, 2, 128, 3, dev)
    o = q.attn_prompt(x, k, v, starts([n], dev))
    check(x, k, v, [n], [n], 1 / math.sqrt(128), o, rows=[0, 1, 127, 128, 2047, 2048, 3000, 4095, 4096, 4099])


def test_many_sequences():
    lens = [(b * 29) % 67 for b in range(150)]
    run(lens, lens, 2, 2, 64, 4)


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("D", [64, 128])
def test_values_at_unseen_places_do_not_matter(value, D):
    """K and V rows of the future, of a neighbouring sequence and of no sequence hold NaN or inf."""
    dev = need_gpu()
    lens = [130, 60, 200]
    n = sum(lens)
    x, k, v = heads(n, 4, D, 1, dev), heads(n + 50, 2, D, 2, dev), heads(n + 50, 2, D, 3, dev)
    k[n:] = value
    v[n:] = value
    k[129], v[129] = value, value                     # the last row of the first sequence
    v[130 + 60 + 150:n] = value                       # the last 50 rows of the last one
    o = q.attn_prompt(x, k, v, starts(lens, dev))
    keep = torch.ones(n, dtype=torch.bool, device=dev)
    keep[129] = False
    keep[130 + 60 + 150:] = False
    # rows that see none of it: within the tolerance of the clean ones' formula
    assert torch.all(torch.isfinite(o[keep].float()))
    check(x[:129], k[:129], v[:129], [129], [129], 1 / math.sqrt(D), o[:129])
    check(x[130:190], k[130:190], v[130:190], [60], [60], 1 / math.sqrt(D), o[130:190])
    check(x[190:340], k[190:340], v[190:340], [150], [150], 1 / math.sqrt(D), o[190:340])


def test_columns_of_a_fused_projection():
    dev = need_gpu()
    H, G, D, lens = 2, 4, 128, [70, 200]
    y = syn.activations(270, (H * G + 2 * H) * D, 2, device=dev)
    x, k, v = (t.view(270, -1, D) for t in y.split([H * G * D, H * D, H * D], dim=1))
    buf = torch.full((270, H * G * D + 8), 3.0, dtype=torch.bfloat16, device=dev)
    out = buf[:, :H * G * D].view(270, H * G, D)
    q.attn_prompt(x, k, v, starts(lens, dev), out=out)
    assert torch.all(buf[:, H * G * D:] == 3.0)
    assert torch.equal(out, q.attn_prompt(x.contiguous(), k.contiguous(), v.contiguous(), starts(lens, dev)))
    check(x, k, v, lens, lens, 1 / math.sqrt(D), out)


@pytest.mark.parametrize("qs,ks", [([0, 40, 90], [0, 40, 90]), ([0, 60, 30], [0, 40, 80]), ([-1, 40, 80], [0, 40, 80]),
                                   ([0, 40, 80], [0, 50, 40]), ([0, 40, 80], [0, 40, 2 ** 31 - 1])])
def test_ranges_that_do_not_hold(qs, ks):
    """Flagged; the sequence that is wrong stays untouched, one that is right is computed."""
    dev = need_gpu()
    x, k, v = heads(80, 2, 64, 1, dev), heads(80, 2, 64, 2, dev), heads(80, 2, 64, 3, dev)
    out = torch.full((80, 2, 64), 4.0, dtype=torch.bfloat16, device=dev)
    st = status(dev)
    t = lambda a: torch.tensor(a, dtype=torch.int32, device=dev)     # noqa: E731
    q.attn_prompt(x, k, v, t(qs), t(ks), out=out, dev_status=st)
    assert read_status(st) == q.ERR_RANGE
    good = [0 <= a[b] <= a[b + 1] <= 80 for a in (qs, ks) for b in range(2)]
    good = [good[0] and good[2], good[1] and good[3]]
    touched = torch.zeros(80, dtype=torch.bool, device=dev)
    for b in range(2):
        if good[b]:
            touched[qs[b]:qs[b + 1]] = True
            n, m = qs[b + 1] - qs[b], ks[b + 1] - ks[b]
            check(x[qs[b]:qs[b + 1]], k[ks[b]:ks[b + 1]], v[ks[b]:ks[b + 1]], [n], [m], 0.125, out[qs[b]:qs[b + 1]])
    assert torch.all(out[~touched] == 4.0)


def test_no_rows():
    dev = need_gpu()
    e = torch.empty((0, 2, 64), dtype=torch.bfloat16, device=dev)
    x = heads(5, 2, 64, 1, dev)
    assert q.attn_prompt(e, e, e, starts([0, 0], dev)).shape == (0, 2, 64)
    o = q.attn_prompt(x, e, e, starts([5], dev), starts([0], dev))
    assert torch.all(o == 0)


def test_the_same_bits_another_stream_and_a_graph():
    dev = need_gpu()
    lens = [300, 77]
    x, k, v = heads(377, 4, 128, 1, dev), heads(377, 2, 128, 2, dev), heads(377, 2, 128, 3, dev)
    cu = starts(lens, dev)
    ref = q.attn_prompt(x, k, v, cu)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        o = q.attn_prompt(x, k, v, cu)
    s.synchronize()
    assert torch.equal(o, ref)
    out = torch.zeros_like(ref)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        q.attn_prompt(x, k, v, cu, out=out)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, ref)


@pytest.mark.parametrize("H,G,D,lens", [(1, 100, 64, [150, 3]), (1, 128, 128, [40, 1]), (1, 131, 64, [70]), (2, 160, 64, [33, 20]),
                                        (1, 65, 128, [9, 260])])
def test_many_heads_to_a_kv_head(H, G, D, lens):
    """One position to a row tile, and heads that are taken in parts."""
    run(lens, lens, H, G, D, 14)


def test_many_sequences_of_two_tiles():
    lens = [(b * 137) % 401 for b in range(40)]
    run(lens, [n + (b * 53) % 90 for b, n in enumerate(lens)], 4, 4, 64, 15)


def test_a_nan_among_heads_taken_in_parts():
    """Rows that see a NaN give NaN, the rows before it what the formula gives."""
    dev = need_gpu()
    n, G, D = 40, 131, 64
    x, k, v = heads(n, G, D, 1, dev), heads(n, 1, D, 2, dev), heads(n, 1, D, 3, dev)
    v[30] = float("nan")
    o = q.attn_prompt(x, k, v, starts([n], dev))
    assert torch.all(torch.isnan(o[30:].float()))
    check(x[:30], k[:30], v[:30], [30], [30], 1 / math.sqrt(D), o[:30])
