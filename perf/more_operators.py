"""The operators of a feed-forward block in FP8 with a scale for each block of 128, as they are measured: the quantisers
of weights and activations, the residual RMSNorm with such scales, the linear, and the gated product (gate and up
projection, SiLU, product and quantisation in one call).

E4M3 codes; a scale of an activation belongs to one token and 128 values, one of a weight to 128 x 128.  Scales of
activations lie as [K / 128][M].  Sizes are those of the package's shapes (Llama-3-8B: hidden 4096, intermediate
14336; Qwen2.5-7B: hidden 3584, intermediate 18944) and of its batch sizes (1, 16, 32) and draft lengths (2, 4, 8).
"""
import math

import torch

own = False

DEV = "cuda"
F8 = torch.float8_e4m3fn
F8_MAX = 448.0
EPS = 1e-5


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # one token in front of the block, batch-1 decode
        {"name": "norm 1x4096", "op": "norm", "M": 1, "K": 4096, "residual": True, "bf16": False},
        # a ragged batch of prompts, with the bf16 output for a W4A16 linear as well
        {"name": "norm 2047x3584 bf16", "op": "norm", "M": 2047, "K": 3584, "residual": True, "bf16": True},
        # attention outputs of a verify pass, 16 sequences, gamma 4, in front of the output projection
        {"name": "quant 80x4096", "op": "quant", "M": 80, "K": 4096},
        # the intermediate values of a batch of prompts, quantised by themselves
        {"name": "quant 4099x14336", "op": "quant", "M": 4099, "K": 14336},
        # a projection whose rows end inside a block
        {"name": "weights 1000x3584", "op": "weights", "N": 1000, "K": 3584},
        # a down projection, once per model load
        {"name": "weights 3584x18944", "op": "weights", "N": 3584, "K": 18944},
        # down projection of one token
        {"name": "linear 1x4096x14336", "op": "linear", "M": 1, "N": 4096, "K": 14336},
        # down projection of the verify rows of 32 sequences, gamma 8
        {"name": "linear 288x3584x18944", "op": "linear", "M": 288, "N": 3584, "K": 18944},
        # down projection of a batch of prompts
        {"name": "linear 8191x4096x14336", "op": "linear", "M": 8191, "N": 4096, "K": 14336},
        # gate and up projection of one token
        {"name": "gated 1x14336x4096", "op": "gated", "M": 1, "N": 14336, "K": 4096, "bf16": False},
        # gate and up projection of the verify rows of 16 sequences, gamma 4, with the bf16 output as well
        {"name": "gated 80x18944x3584 bf16", "op": "gated", "M": 80, "N": 18944, "K": 3584, "bf16": True},
        # gate and up projection of a batch of prompts
        {"name": "gated 8192x14336x4096", "op": "gated", "M": 8192, "N": 14336, "K": 4096, "bf16": False},
    ]


def _spread(rng, lo, hi):
    """A whole number in [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


BLOCKS = [1, 2, 3, 5, 8, 11, 16, 20, 28, 32, 37, 40, 56, 64, 80, 112, 148]      # sizes in blocks of 128
MOST = 8191 * 4096 * 14336                                                    # products of the largest linear


def draw(rng):
    op = rng.choice(["norm", "quant", "weights", "linear", "linear", "gated", "gated"])
    K = 128 * rng.choice(BLOCKS)
    if op == "norm":
        return {"op": op, "M": _spread(rng, 1, min(8192, 8192 * 4096 // K)), "K": K, "residual": rng.random() < 0.7,
                "bf16": rng.random() < 0.4}
    if op == "quant":
        return {"op": op, "M": _spread(rng, 1, min(8192, 4099 * 14336 // K)), "K": K}
    if op == "weights":
        return {"op": op, "N": _spread(rng, 1, min(18944, 3584 * 18944 // K)), "K": K}
    if op == "linear":
        N = _spread(rng, 1, 18944) if rng.random() < 0.5 else 128 * rng.choice(BLOCKS)
        return {"op": op, "M": _spread(rng, 1, min(8192, MOST // (N * K))), "N": N, "K": K}
    N = 128 * rng.choice(BLOCKS)
    return {"op": op, "M": _spread(rng, 1, min(8192, MOST // (2 * N * K))), "N": N, "K": K, "bf16": rng.random() < 0.4}


def work(case):
    op, K = case["op"], case["K"]
    if op == "weights":
        N = case["N"]
        return {"bytes": 3 * N * K + 4 * (-(-N // 128)) * (K // 128), "flops": 4 * N * K}
    M = case["M"]
    scales = 4 * M * (K // 128)
    if op == "quant":
        return {"bytes": 3 * M * K + scales, "flops": 4 * M * K}
    if op == "norm":
        return {"bytes": M * K * (2 + (4 if case["residual"] else 0) + 1 + (2 if case["bf16"] else 0)) + scales + 2 * K, "flops": 8 * M * K}
    N = case["N"]
    if op == "linear":
        return {"bytes": M * K + N * K + scales + 4 * (-(-N // 128)) * (K // 128) + 2 * M * N, "flops": 2 * M * N * K}
    return {"bytes": M * K + 2 * N * K + scales + 8 * (N // 128) * (K // 128) + M * N * (3 if case["bf16"] else 1) + 4 * M * (N // 128),
            "flops": 4 * M * N * K + 8 * M * N}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _rows(M, K, g):
    """Activations: N(0, 1), one channel in 100 twenty times as large, tokens of different sizes."""
    x = torch.randn((M, K), generator=g, device=DEV)
    x[:, 3::100] *= 20.0
    return x * (0.5 + torch.rand((M, 1), generator=g, device=DEV))


def _matrix(N, K, g):
    """Weights: N(0, 1 / K), rows of different sizes."""
    return torch.randn((N, K), generator=g, device=DEV) * (0.5 + torch.rand((N, 1), generator=g, device=DEV)) / math.sqrt(K)


def _codes_of_rows(x):
    """E4M3 codes and [K / 128][M] scales of activations."""
    M, K = x.shape
    b = x.view(M, K // 128, 128)
    s = b.abs().amax(-1).float() / F8_MAX
    c = (b / torch.where(s > 0, s, torch.ones_like(s))[..., None]).clamp(-F8_MAX, F8_MAX).to(F8).view(M, K)
    return c, s.t().contiguous()


def _codes_of_matrix(w):
    """E4M3 codes and [ceil(N / 128)][K / 128] scales of weights."""
    N, K = w.shape
    top = w.abs().view(N, K // 128, 128).amax(-1)
    n = -(-N // 128)
    s = torch.zeros((n * 128, K // 128), device=DEV)
    s[:N] = top
    s = s.view(n, 128, K // 128).amax(1) / F8_MAX
    each = s.repeat_interleave(128, 0)[:N]
    c = (w.view(N, K // 128, 128) / torch.where(each > 0, each, torch.ones_like(each))[..., None]).clamp(-F8_MAX, F8_MAX)
    return c.to(F8).view(N, K), s


def prepare(case, seed):
    g = _gen(seed)
    op, K = case["op"], case["K"]
    s = {"case": case, "status": torch.zeros(1, dtype=torch.int32, device=DEV)}
    if op == "weights":
        s["w"] = _matrix(case["N"], K, g).to(torch.float16)
        return s
    M = case["M"]
    x = _rows(M, K, g)
    if op in ("norm", "quant"):
        s["x"] = x.to(torch.bfloat16)
        if op == "norm":
            if case["residual"]:
                s["r"] = (torch.randn((M, K), generator=g, device=DEV) * 2.0).to(torch.bfloat16)
            s["w"] = (1.0 + 0.1 * torch.randn((K,), generator=g, device=DEV)).to(torch.bfloat16)
        return s
    s["xq"], s["sa"] = _codes_of_rows(x)
    for name in ("g", "u") if op == "gated" else ("w",):
        s[name], s["s" + name] = _codes_of_matrix(_matrix(case["N"], K, g))
    return s


# ---------------------------------------------------------------------------
# the framework's kernels
# ---------------------------------------------------------------------------
def _codes(s, name, rows, cols):
    """A buffer of codes that a program keeps, as the library takes it and as the values it stands for."""
    s[name] = torch.empty((rows, cols), dtype=torch.uint8, device=DEV)
    return s[name].view(F8)


def _kept(s):
    """The buffers that a program keeps for its layers, and the list of the outputs."""
    case = s["case"]
    op, K = case["op"], case["K"]
    if op == "weights":
        n = -(-case["N"] // 128)
        s["sw"] = torch.empty((n, K // 128), dtype=torch.float32, device=DEV)
        return [_codes(s, "w8", case["N"], K), s["sw"]]
    M = case["M"]
    if op == "linear":
        s["xb"], s["wb"] = s["xq"].view(torch.uint8), s["w"].view(torch.uint8)
        s["y"] = torch.empty((M, case["N"]), dtype=torch.bfloat16, device=DEV)
        return s["y"]
    if op == "gated":
        s["xb"], s["gb"], s["ub"] = (s[i].view(torch.uint8) for i in ("xq", "g", "u"))
        s["sh"] = torch.empty((case["N"] // 128, M), dtype=torch.float32, device=DEV)
        s["y"] = torch.empty((M, case["N"]), dtype=torch.bfloat16, device=DEV) if case["bf16"] else None
        return [_codes(s, "hq", M, case["N"]), s["sh"]] + ([s["y"]] if case["bf16"] else [])
    s["so"] = torch.empty((K // 128, M), dtype=torch.float32, device=DEV)
    out = [_codes(s, "xq", M, K), s["so"]]
    if op == "quant":
        return out
    s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
    s["y"] = torch.empty_like(s["x"]) if case["bf16"] else None
    return out + [s[i] for i in ("h", "y") if s[i] is not None]


def _run_own(s):
    from quantized_speculative_decoding_shared_gb300 import binding as q
    case, st = s["case"], s["status"]
    if "out" not in s:
        s["out"] = _kept(s)
    op, K = case["op"], case["K"]
    if op == "weights":
        rc = q.qspec_quant_weights_fp8_block(s["w"], case["N"], K, s["w8"], s["sw"], st)
    elif op == "quant":
        rc = q.qspec_quant_act_fp8_block(s["x"], case["M"], K, K, s["xq"], s["so"], case["M"], st)
    elif op == "norm":
        rc = q.qspec_rmsnorm_fp8_block(s["x"], K, s.get("r"), K, s["w"], EPS, case["M"], K, s["h"], K, s["xq"], s["so"], case["M"],
                                       s["y"], K, st)
    elif op == "linear":
        rc = q.qspec_linear_fp8_block(s["xb"], s["sa"], case["M"], s["wb"], s["sw"], case["M"], case["N"], K, s["y"], case["N"], st)
    else:
        rc = q.qspec_gated_fp8_block(s["xb"], s["sa"], case["M"], s["gb"], s["sg"], s["ub"], s["su"], case["M"], case["N"], K,
                                     s["hq"], s["sh"], case["M"], s["y"], case["N"], st)
    assert rc == q.OK, rc
    return s["out"]


# ---------------------------------------------------------------------------
# the plain forms, in 32 bits
# ---------------------------------------------------------------------------
def _plain_rows(xq, sa):
    """The values that codes and scales of activations stand for."""
    M, K = xq.shape
    return (xq.float().view(M, K // 128, 128) * sa.t()[..., None]).view(M, K)


def _plain_matrix(w8, sw):
    """The values that codes and scales of weights stand for."""
    N, K = w8.shape
    return (w8.float().view(N, K // 128, 128) * sw.repeat_interleave(128, 0)[:N, :, None]).view(N, K)


def _run_plain(s):
    case, op = s["case"], s["case"]["op"]
    if op == "weights":
        return list(_codes_of_matrix(s["w"].float()))
    if op == "quant":
        return list(_codes_of_rows(s["x"].float()))
    if op == "norm":
        h, out = s["x"].float(), []
        if case["residual"]:
            hb = (h + s["r"].float()).to(torch.bfloat16)
            h = hb.float()
            out.append(hb)
        y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["w"].float()
        return list(_codes_of_rows(y)) + out + ([y.to(torch.bfloat16)] if case["bf16"] else [])
    x = _plain_rows(s["xq"], s["sa"])
    if op == "linear":
        return torch.matmul(x, _plain_matrix(s["w"], s["sw"]).t()).to(torch.bfloat16)
    a = torch.matmul(x, _plain_matrix(s["g"], s["sg"]).t())
    h = a / (1.0 + torch.exp(-a)) * torch.matmul(x, _plain_matrix(s["u"], s["su"]).t())
    return list(_codes_of_rows(h)) + ([h.to(torch.bfloat16)] if case["bf16"] else [])


def run(state):
    return _run_own(state) if own else _run_plain(state)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_codes(y):
    """Rows [M][K] -> y over its block's scale, and the scales [K / 128][M]."""
    parts = y.double().split(128, dim=1)
    tops = [p.abs().max(dim=1).values / F8_MAX for p in parts]
    return [torch.cat([p / torch.where(t > 0, t, 1.0).unsqueeze(1) for p, t in zip(parts, tops)], dim=1), torch.stack(tops)]


def _exact_product(xq, sa, w8, sw):
    """The sum over blocks of 128: scales times the product of the codes."""
    y = torch.zeros((xq.shape[0], w8.shape[0]), dtype=torch.float64, device=DEV)
    of = torch.arange(w8.shape[0], device=DEV) // 128
    for i in range(sa.shape[0]):
        a = xq[:, 128 * i:128 * i + 128].double() * sa[i].double().unsqueeze(1)
        b = w8[:, 128 * i:128 * i + 128].double() * sw[of, i].double().unsqueeze(1)
        y.addmm_(a, b.T)
    return y


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "weights":
        w, cols, tops = s["w"].double(), [], []
        for at in range(0, case["N"], 128):
            c, t = _exact_codes(w[at:at + 128])
            t = t.max(dim=1).values
            by = torch.where(t > 0, t, 1.0).repeat_interleave(128)
            cols.append(w[at:at + 128] / by)
            tops.append(t)
        return [torch.cat(cols), torch.stack(tops)]
    if op == "quant":
        return _exact_codes(s["x"])
    if op == "norm":
        x, out = s["x"].double(), []
        if case["residual"]:
            x = x + s["r"].double()
            out.append(x)
            x = x.to(torch.bfloat16).double()
        y = x / torch.sqrt(x.pow(2).sum(-1, keepdim=True) / case["K"] + EPS) * s["w"].double()
        return _exact_codes(y) + out + ([y] if case["bf16"] else [])
    if op == "linear":
        return _exact_product(s["xq"], s["sa"], s["w"], s["sw"])
    a = _exact_product(s["xq"], s["sa"], s["g"], s["sg"])
    h = a * torch.sigmoid(a) * _exact_product(s["xq"], s["sa"], s["u"], s["su"])
    return _exact_codes(h) + ([h] if case["bf16"] else [])
