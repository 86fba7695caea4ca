"""Rows into and out of the 4-bit cache where the ranges of some sequences do not hold: those are flagged and left
untouched, every other sequence's rows arrive, wherever the starts lead a search."""
import pytest
import torch

from quantized_speculative_decoding_shared_gb300 import binding as q, synthetic as syn
from gpuhelp import need_gpu, read_status, status
from layerref import pack, quantise_rows, values, words

pytestmark = pytest.mark.gpu


def ints(v, dev):
    return torch.tensor(v, dtype=torch.int32, device=dev)


def one_bad_start(B):
    """One row to a sequence; the start in the middle is far too large, which spoils two of them."""
    start = list(range(B + 1))
    start[B // 2] = 10 ** 6
    return start


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("start,rows", [([0, 9, 3, 8], 8), ([0, 4, 100, 8, 12], 12), ([50, 0, 4, 8, -1, 8, 11], 11),
                                        ([0, 300, 40, 170], 200), (one_bad_start(40), 40), (one_bad_start(1024), 1024),
                                        (one_bad_start(1500), 1500)])
def test_the_other_sequences_rows(start, rows, D):
    dev = need_gpu()
    B, H, T = len(start) - 1, 2, 160
    valid = [0 <= a <= b <= rows and b - a + 3 <= T for a, b in zip(start, start[1:])]
    assert not all(valid) and any(valid)
    k, v = (syn.activations(rows * H, D, i, device=dev).view(rows, H, D) for i in (1, 2))
    cache = q.kv4_cache(B, H, T, D, device=dev)
    for t in cache:
        t.fill_(0x5A)
    want = [t.clone() for t in cache]
    for b in range(B):
        if valid[b]:
            n = start[b + 1] - start[b]
            for x, codes, sz in ((k, want[0], want[1]), (v, want[2], want[3])):
                c, s, z = quantise_rows(x[start[b]:start[b + 1]])
                codes[b, :, 3:3 + n] = pack(c).transpose(0, 1)
                sz[b, :, 3:3 + n] = words(s, z).transpose(0, 1)
    st = status(dev)
    q.kv4_append(cache, k, v, ints(start, dev), ints([3] * B, dev), dev_status=st)
    assert read_status(st) == q.ERR_RANGE
    for got, ref in zip(cache, want):
        assert torch.equal(got, ref)
    st = status(dev)
    ko, vo = q.kv4_load(cache, ints(start, dev), ints([3] * B, dev), rows, dev_status=st)
    assert read_status(st) == q.ERR_RANGE
    rk, rv = torch.zeros_like(k), torch.zeros_like(v)
    for b in range(B):
        if valid[b]:
            n = start[b + 1] - start[b]
            for o, codes, sz in ((rk, want[0], want[1]), (rv, want[2], want[3])):
                o[start[b]:start[b + 1]] = values(codes[b, :, 3:3 + n], sz[b, :, 3:3 + n]).transpose(0, 1).to(torch.bfloat16)
    assert torch.equal(ko, rk) and torch.equal(vo, rv)
