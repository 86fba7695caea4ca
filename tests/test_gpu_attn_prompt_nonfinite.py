"""Prompt attention with values that are not finite at places that rows see: each row gives what the formula gives, at
a cost that stays near the clean call's.  Tolerances as in test_gpu_attn_prompt.py."""
import math

import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q
from gpuhelp import need_gpu, read_status, status
from test_gpu_attn_prompt import check, heads, starts

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


def inputs(n, H, G, D, dev):
    return heads(n, H * G, D, 1, dev), heads(n, H, D, 2, dev), heads(n, H, D, 3, dev)


def call(x, k, v, cu, scale=None):
    st = status(x.device)
    o = q.attn_prompt(x, k, v, cu, scale=scale, dev_status=st)
    assert read_status(st) == 0
    return o


def seconds(f):
    """The shortest of three calls, after one."""
    f()
    best = INF
    for _ in range(3):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        f()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b) * 1e-3)
    return best


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G,lens", [(4, [700]), (7, [300, 1, 411]), (1, [129, 520])])
def test_one_dimension_of_an_early_v_row(D, G, lens):
    """Rows that see it: NaN in that dimension, the formula in the others."""
    dev = need_gpu()
    n = sum(lens)
    x, k, v = inputs(n, 2, G, D, dev)
    v[1, 1, 5] = NAN
    o = call(x, k, v, starts(lens, dev))
    poisoned = torch.zeros_like(o, dtype=torch.bool)
    poisoned[1:lens[0], G:, 5] = True
    assert torch.equal(torch.isnan(o.float()), poisoned)
    clean = v.clone()
    clean[1, 1, 5] = 0
    check(x, k, clean, lens, lens, 1 / math.sqrt(D), o.where(~poisoned, call(x, k, clean, starts(lens, dev))))


@pytest.mark.parametrize("D", [64, 128])
def test_seen_by_some_and_not_by_others(D):
    """A NaN that a row sees, in one dimension, and one that it does not see, in another."""
    dev = need_gpu()
    n, G = 450, 4
    x, k, v = inputs(n, 1, G, D, dev)
    clean = v.clone()
    v[200, 0, 3] = NAN
    v[n - 1, 0, 7] = NAN
    v[n - 60, 0, :] = INF
    o = call(x, k, v, starts([n], dev))
    at = torch.arange(n, device=dev)
    bad = torch.zeros((n, G, D), dtype=torch.bool, device=dev)
    bad[at >= 200, :, 3] = True
    bad[at >= n - 60] = True
    assert torch.equal(~torch.isfinite(o.float()), bad)
    check(x, k, clean, [n], [n], 1 / math.sqrt(D), o.where(~bad, call(x, k, clean, starts([n], dev))))


@pytest.mark.parametrize("at", [1, 200, 699])
def test_a_key_that_is_nan(at):
    dev = need_gpu()
    n, D = 700, 128
    x, k, v = inputs(n, 2, 2, D, dev)
    k[at, 0, 9] = NAN
    o = call(x, k, v, starts([n], dev))
    assert torch.isnan(o[at:, :2].float()).all() and torch.isfinite(o[:at].float()).all() and torch.isfinite(o[:, 2:].float()).all()
    check(x[:at], k[:at], v[:at], [at], [at], 1 / math.sqrt(D), o[:at])


@pytest.mark.parametrize("at", [0, 1, 200, 699])
@pytest.mark.parametrize("value", [INF, -INF])
def test_a_key_that_is_infinite(value, at):
    """Rows whose score of it is plus infinity have no softmax; where it is minus infinity it weighs nothing."""
    dev = need_gpu()
    n, D = 700, 64
    x, k, v = inputs(n, 1, 2, D, dev)
    x[:, :, 9] = torch.where(x[:, :, 9] == 0, torch.ones_like(x[:, :, 9]), x[:, :, 9])
    k[at, 0, 9] = value
    o = call(x, k, v, starts([n], dev))
    sees = (torch.arange(n, device=dev) >= at)[:, None]
    plus = sees & (x[:, :, 9].float() * (1.0 if value > 0 else -1.0) > 0)
    assert torch.isnan(o.float())[plus].all()
    far = k.clone()
    far[at, 0] = 0
    far[at, 0, 9] = math.copysign(1e30, value)                  # the same weight of nothing where the score is below
    for j in range(2):
        keep = ~plus[:, j]
        if at == 0:
            keep = keep & (torch.arange(n, device=dev) > 0)     # (a row of one key has that key alone)
        a = ((x[:, j].double() @ far[:, 0].double().T) / math.sqrt(D)).masked_fill(
            torch.arange(n, device=dev)[None, :] > torch.arange(n, device=dev)[:, None], -INF)
        p = torch.softmax(a, -1)
        ref, A = p @ v[:, 0].double(), p @ v[:, 0].double().abs()
        top = (x[:, j].double().abs() @ k[:, 0].double().abs().nan_to_num(posinf=0).T).amax(-1, keepdim=True)
        tol = (2.0 ** -8 + 2.0 ** -12 + 2 * 16 * 2.0 ** -24 / math.sqrt(D) * top) * A + 2.0 ** -8 * ref.abs() + 1e-30
        assert torch.all(((o[:, j].double() - ref).abs() <= tol)[keep])


@pytest.mark.parametrize("at", [130, 300, 511])
def test_a_score_far_above_all_before_it(at):
    """Within one key tile the scores pass the reference by more than fp32 holds."""
    dev = need_gpu()
    n, D = 600, 64
    x, k, v = inputs(n, 1, 2, D, dev)
    x = x.abs().clamp(min=0.01)
    k[at] = 40.0
    o = call(x, k, v, starts([n], dev))
    check(x, k, v, [n], [n], 1 / math.sqrt(D), o)


@pytest.mark.parametrize("what,at", [("v", 1), ("v", 2000), ("v", slice(1000, 4096)), ("k", 1), ("k", 2000)])
def test_the_cost_of_a_value_that_is_not_finite(what, at):
    """4096 rows that nearly all see a NaN (V) or an infinity (K): within 30 times the clean call, where a walk over the
    keys for each row took 1000 times."""
    dev = need_gpu()
    n = 4096
    x, k, v = inputs(n, 8, 4, 128, dev)
    cu = starts([n], dev)
    out = torch.empty_like(x)
    clean = seconds(lambda: q.attn_prompt(x, k, v, cu, out=out))
    if what == "v":
        v[at] = NAN
    else:
        k[at, :, 17] = INF
    assert seconds(lambda: q.attn_prompt(x, k, v, cu, out=out)) <= 30 * clean
