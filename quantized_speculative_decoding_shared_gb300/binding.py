"""Thin Python binding of libqspec.so (the C ABI in include/qspec.h).

Argument marshalling only: every step of the hot path runs in the library's
CUDA kernels.  PyTorch supplies device memory and streams.  The functions
named ``qspec_*`` mirror the C calls one to one (caller-provided outputs);
the short names (``pack_weights`` ...) allocate the outputs with torch and
call the same entry points.

There is no fallback: if libqspec.so is missing or the device is not an
sm_103 part, the calls raise.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(HERE, "_lib", "libqspec.so")

GROUP = 128
MAX_GAMMA = 16
STATUS = {0: "QSPEC_OK", 1: "QSPEC_ERR_NULL", 2: "QSPEC_ERR_SHAPE", 3: "QSPEC_ERR_ALIGN",
          4: "QSPEC_ERR_LAUNCH", 5: "QSPEC_ERR_WORKSPACE", 6: "QSPEC_ERR_RANGE",
          7: "QSPEC_ERR_ZERO_POINT", 8: "QSPEC_ERR_NONFINITE", 9: "QSPEC_ERR_TIMEOUT",
          10: "QSPEC_ERR_UNSUPPORTED"}
OK, ERR_NULL, ERR_SHAPE, ERR_ALIGN, ERR_LAUNCH, ERR_WORKSPACE = 0, 1, 2, 3, 4, 5
ERR_RANGE, ERR_ZERO_POINT, ERR_NONFINITE, ERR_TIMEOUT, ERR_UNSUPPORTED = 6, 7, 8, 9, 10

EXPORTED = ["qspec_version", "qspec_status_string", "qspec_last_cuda_error", "qspec_kernel_launches",
            "qspec_pack_weights",
            "qspec_quant_act_int4", "qspec_linear_w4a4", "qspec_linear_w4a4_bf16", "qspec_linear_w4a16",
            "qspec_verify_workspace_bytes", "qspec_verify_greedy", "qspec_verify_sample",
            "qspec_kv_overwrite", "qspec_verify_sample_noalloc", "qspec_draft_workspace_bytes",
            "qspec_draft_sample", "qspec_debug_linear_bounded", "qspec_quant_weights_fp8",
            "qspec_quant_act_fp8", "qspec_linear_fp8", "qspec_linear_w4a16_kv",
            "qspec_rmsnorm_fp8", "qspec_kv4_append", "qspec_kv4_load", "qspec_attn_kv4_workspace_bytes",
            "qspec_attn_kv4", "qspec_attn_prompt", "qspec_debug_attn_kv4_bounded",
            "qspec_debug_attn_prompt_bounded"]
KERNEL_W4A16_TC, KERNEL_W4A4_GEMV_TC, KERNEL_W4A4_TC = 0, 1, 2
NOALLOC_SCRATCH_BYTES = 1 << 20


class QspecError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str = ""):
        self.status = status
        msg = "%s failed: %s" % (where, STATUS.get(status, str(status)))
        if detail:
            msg += " (%s)" % detail
        super().__init__(msg)


_lock = threading.Lock()
_lib = None


def load_library(path: str | None = None) -> ctypes.CDLL:
    """Load libqspec.so and declare its prototypes.  Raises if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    with _lock:
        if _lib is not None and path is None:
            return _lib
        p = path or LIB_PATH
        if not os.path.exists(p):
            raise RuntimeError("libqspec.so is not built (%s); run "
                               "quantized_speculative_decoding_shared_gb300.build.build()" % p)
        lib = ctypes.CDLL(p)
        vp, i32, sz_t, u64 = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_uint64
        f32 = ctypes.c_float
        proto = {
            "qspec_version": ([], i32),
            "qspec_kernel_launches": ([], ctypes.c_ulonglong),
            "qspec_status_string": ([i32], ctypes.c_char_p),
            "qspec_last_cuda_error": ([], ctypes.c_char_p),
            "qspec_pack_weights": ([vp, vp, vp, i32, i32, vp, vp, vp, vp], i32),
            "qspec_quant_act_int4": ([vp, i32, i32, i32, vp, vp, vp, vp, vp], i32),
            "qspec_linear_w4a4": ([vp, vp, vp, vp, vp, i32, i32, i32, vp, i32, vp, vp, vp], i32),
            "qspec_linear_w4a4_bf16": ([vp, i32, vp, vp, i32, i32, i32, vp, i32, vp, vp, vp, vp, vp, vp],
                                       i32),
            "qspec_linear_w4a16": ([vp, i32, vp, vp, i32, i32, i32, vp, i32, vp, vp], i32),
            "qspec_verify_workspace_bytes": ([i32, i32, i32], sz_t),
            "qspec_verify_greedy": ([vp, vp, i32, i32, i32, vp, vp, vp, sz_t, vp, vp], i32),
            "qspec_verify_sample": ([vp, vp, vp, i32, i32, i32, u64, u64, vp, vp, vp, sz_t, vp, vp],
                                    i32),
            "qspec_kv_overwrite": ([vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, vp, vp],
                                   i32),
            "qspec_verify_sample_noalloc": ([vp, vp, vp, i32, i32, i32, u64, u64, vp, vp, vp, vp],
                                            i32),
            "qspec_draft_workspace_bytes": ([i32, i32], sz_t),
            "qspec_draft_sample": ([vp, i32, i32, u64, u64, i32, vp, vp, vp, vp, sz_t, vp, vp], i32),
            "qspec_debug_linear_bounded": ([i32, vp, vp, vp, vp, vp, vp, i32, i32, i32, vp, i32,
                                            ctypes.c_uint32, i32, vp, vp], i32),
            "qspec_quant_weights_fp8": ([vp, i32, i32, vp, vp, vp, vp], i32),
            "qspec_quant_act_fp8": ([vp, i32, i32, i32, vp, vp, vp, vp], i32),
            "qspec_linear_fp8": ([vp, vp, vp, vp, i32, i32, i32, vp, i32, vp, vp], i32),
            "qspec_linear_w4a16_kv": ([vp, i32, vp, vp, i32, i32, i32, vp, i32, i32, i32, i32, i32, i32,
                                       vp, vp, vp, vp, vp, vp], i32),
            "qspec_rmsnorm_fp8": ([vp, i32, vp, i32, vp, f32, i32, i32, vp, i32, vp, vp, vp, i32, vp, vp], i32),
            "qspec_kv4_append": ([vp, i32, vp, i32, vp, vp, i32, i32, i32, i32, i32, vp, vp, vp, vp, vp, vp],
                                 i32),
            "qspec_kv4_load": ([vp, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, vp, i32, vp, i32, vp, vp], i32),
            "qspec_attn_kv4_workspace_bytes": ([i32, i32, i32, i32, i32], sz_t),
            "qspec_attn_kv4": ([vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp, i32, vp, sz_t,
                                vp, vp], i32),
            "qspec_attn_prompt": ([vp, i32, vp, i32, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp, i32,
                                   vp, vp], i32),
            "qspec_debug_attn_kv4_bounded": ([vp, i32, vp, vp, vp, vp, vp, i32, i32, i32, i32, i32, i32, f32, vp, i32,
                                              vp, sz_t, ctypes.c_uint32, i32, vp, vp], i32),
            "qspec_debug_attn_prompt_bounded": ([vp, i32, vp, i32, vp, i32, vp, vp, i32, i32, i32, i32, i32, i32, f32,
                                                 vp, i32, ctypes.c_uint32, i32, vp, vp], i32),
        }
        for name, (args, res) in proto.items():
            f = getattr(lib, name)
            f.argtypes = args
            f.restype = res
        if path is None:
            _lib = lib
        return lib


def _ptr(t):
    # a plain int: the declared argument types make it a pointer, and a
    # c_void_p object per argument costs as much as the rest of a small call
    return None if t is None else t.data_ptr()


def _stream(stream):
    if stream is None:
        # the handle alone (building a torch.cuda.Stream object takes 3 us)
        if not torch.cuda.is_initialized():
            torch.cuda.init()
        return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())
    return stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)


def on_stream(stream):
    """The context in which what a call on `stream` (None, a torch stream or a raw handle) makes and fills belongs to
    that stream: torch orders a fill, and hands freed memory out again, by the stream that was current."""
    if stream is None:
        return contextlib.nullcontext()
    if not isinstance(stream, torch.cuda.Stream):
        handle = _stream(stream)
        stream = torch.cuda.ExternalStream(0 if handle == 1 else handle)    # (1: the legacy default stream by name)
    return torch.cuda.stream(stream)


def _allocates(call):
    """A call that makes tensors: with `stream` given they are made on it (memory of the current stream's pool may still
    be written by work queued there, and what a call drops on return would go back to that pool too early)."""
    place = call.__code__.co_varnames.index("stream")

    @functools.wraps(call)
    def made(*args, **kw):
        stream = args[place] if len(args) > place else kw.get("stream")
        if stream is None:
            return call(*args, **kw)
        with on_stream(stream):
            return call(*args, **kw)
    return made


def _check(rc: int, where: str):
    if rc != OK:
        detail = ""
        if rc == ERR_LAUNCH:
            detail = load_library().qspec_last_cuda_error().decode()
        raise QspecError(rc, where, detail)


def _need(t, dtype, name):
    if t.device.type != "cuda":
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dtype != dtype:
        raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


# ---------------------------------------------------------------------------
# one-to-one wrappers of the C calls (outputs provided by the caller)
# ---------------------------------------------------------------------------
def qspec_pack_weights(codes, s, z, N, K, packed, sz, dev_status=None, stream=None):
    return load_library().qspec_pack_weights(_ptr(codes), _ptr(s), _ptr(z), N, K, _ptr(packed),
                                             _ptr(sz), _ptr(dev_status), _stream(stream))


def qspec_quant_act_int4(x, M, K, ldx, xq, sx, qs, dev_status=None, stream=None):
    return load_library().qspec_quant_act_int4(_ptr(x), M, K, ldx, _ptr(xq), _ptr(sx), _ptr(qs),
                                               _ptr(dev_status), _stream(stream))


def qspec_linear_w4a4(xq, sx, qs, packed, sz, M, N, K, y, ldy, dbg_I=None, dev_status=None,
                      stream=None):
    return load_library().qspec_linear_w4a4(_ptr(xq), _ptr(sx), _ptr(qs), _ptr(packed), _ptr(sz),
                                            M, N, K, _ptr(y), ldy, _ptr(dbg_I), _ptr(dev_status),
                                            _stream(stream))


def qspec_linear_w4a4_bf16(x, ldx, packed, sz, M, N, K, y, ldy, xq, sx, qs, dbg_I=None,
                           dev_status=None, stream=None):
    return load_library().qspec_linear_w4a4_bf16(_ptr(x), ldx, _ptr(packed), _ptr(sz), M, N, K,
                                                 _ptr(y), ldy, _ptr(xq), _ptr(sx), _ptr(qs),
                                                 _ptr(dbg_I), _ptr(dev_status), _stream(stream))


def qspec_linear_w4a16(x, ldx, packed, sz, M, N, K, y, ldy, dev_status=None, stream=None):
    return load_library().qspec_linear_w4a16(_ptr(x), ldx, _ptr(packed), _ptr(sz), M, N, K,
                                             _ptr(y), ldy, _ptr(dev_status), _stream(stream))


def qspec_linear_w4a16_kv(x, ldx, packed, sz, M, N, K, y, ldy, kv_col0, H, D, T, gamma, k_cache, v_cache,
                          base_pos, n_acc, dev_status=None, stream=None):
    return load_library().qspec_linear_w4a16_kv(_ptr(x), ldx, _ptr(packed), _ptr(sz), M, N, K, _ptr(y), ldy,
                                                kv_col0, H, D, T, gamma, _ptr(k_cache), _ptr(v_cache),
                                                _ptr(base_pos), _ptr(n_acc), _ptr(dev_status), _stream(stream))


def qspec_verify_workspace_bytes(B, gamma, V):
    return int(load_library().qspec_verify_workspace_bytes(B, gamma, V))


def qspec_verify_greedy(p, draft, B, gamma, V, n_acc, out, workspace, ws_bytes, dev_status=None,
                        stream=None):
    return load_library().qspec_verify_greedy(_ptr(p), _ptr(draft), B, gamma, V, _ptr(n_acc),
                                              _ptr(out), _ptr(workspace), ws_bytes,
                                              _ptr(dev_status), _stream(stream))


def qspec_verify_sample(p, q, draft, B, gamma, V, seed, rnd, n_acc, out, workspace, ws_bytes,
                        dev_status=None, stream=None):
    return load_library().qspec_verify_sample(_ptr(p), _ptr(q), _ptr(draft), B, gamma, V,
                                              ctypes.c_uint64(seed), ctypes.c_uint64(rnd),
                                              _ptr(n_acc), _ptr(out), _ptr(workspace), ws_bytes,
                                              _ptr(dev_status), _stream(stream))


def qspec_verify_sample_noalloc(p, q, draft, B, gamma, V, seed, rnd, n_acc, out, dev_status=None,
                                stream=None):
    """Sampled verification with the library's built-in scratch array: for
    callers that cannot allocate device memory (see include/qspec.h)."""
    return load_library().qspec_verify_sample_noalloc(_ptr(p), _ptr(q), _ptr(draft), B, gamma, V,
                                                      ctypes.c_uint64(seed), ctypes.c_uint64(rnd),
                                                      _ptr(n_acc), _ptr(out), _ptr(dev_status),
                                                      _stream(stream))


def qspec_draft_workspace_bytes(B, V):
    return int(load_library().qspec_draft_workspace_bytes(B, V))


def qspec_draft_sample(q, B, V, seed, rnd, step, token, confidence, entropy, workspace, ws_bytes,
                       dev_status=None, stream=None):
    return load_library().qspec_draft_sample(_ptr(q), B, V, ctypes.c_uint64(seed), ctypes.c_uint64(rnd),
                                             step, _ptr(token), _ptr(confidence), _ptr(entropy),
                                             _ptr(workspace), ws_bytes, _ptr(dev_status), _stream(stream))


def qspec_kv_overwrite(k_cache, v_cache, k_new, v_new, base_pos, n_acc, L, B, H, T, D, gamma,
                       dev_status=None, stream=None):
    return load_library().qspec_kv_overwrite(_ptr(k_cache), _ptr(v_cache), _ptr(k_new),
                                             _ptr(v_new), _ptr(base_pos), _ptr(n_acc), L, B, H, T,
                                             D, gamma, _ptr(dev_status), _stream(stream))


def qspec_kernel_launches():
    """Kernel launches this library has issued (graph captures count once)."""
    return int(load_library().qspec_kernel_launches())


def qspec_debug_linear_bounded(kernel, x, xq, sx, qs, packed, sz, M, N, K, y, ldy, wait_limit,
                               stall, dev_status=None, stream=None):
    """Test diagnostic: one tensor-core linear kernel with a chosen bound on
    its barrier waits (and, with stall, a wait made to run out)."""
    return load_library().qspec_debug_linear_bounded(kernel, _ptr(x), _ptr(xq), _ptr(sx), _ptr(qs),
                                                     _ptr(packed), _ptr(sz), M, N, K, _ptr(y), ldy,
                                                     ctypes.c_uint32(wait_limit), stall,
                                                     _ptr(dev_status), _stream(stream))


def qspec_quant_weights_fp8(w16, N, K, w8, s8, dev_status=None, stream=None):
    return load_library().qspec_quant_weights_fp8(_ptr(w16), N, K, _ptr(w8), _ptr(s8), _ptr(dev_status),
                                                  _stream(stream))


def qspec_quant_act_fp8(x, M, K, ldx, xq, sa, dev_status=None, stream=None):
    return load_library().qspec_quant_act_fp8(_ptr(x), M, K, ldx, _ptr(xq), _ptr(sa), _ptr(dev_status),
                                              _stream(stream))


def qspec_linear_fp8(xq, sa, w8, s8, M, N, K, y, ldy, dev_status=None, stream=None):
    return load_library().qspec_linear_fp8(_ptr(xq), _ptr(sa), _ptr(w8), _ptr(s8), M, N, K, _ptr(y), ldy,
                                           _ptr(dev_status), _stream(stream))


def qspec_rmsnorm_fp8(x, ldx, res, ldr, w, eps, M, K, h, ldh, xq, sa, y, ldy, dev_status=None, stream=None):
    return load_library().qspec_rmsnorm_fp8(_ptr(x), ldx, _ptr(res), ldr, _ptr(w), eps, M, K, _ptr(h), ldh,
                                            _ptr(xq), _ptr(sa), _ptr(y), ldy, _ptr(dev_status), _stream(stream))


def qspec_kv4_append(k, ldk, v, ldv, row_start, base_pos, rows, B, H, T, D, k_codes, k_sz, v_codes, v_sz,
                     dev_status=None, stream=None):
    return load_library().qspec_kv4_append(_ptr(k), ldk, _ptr(v), ldv, _ptr(row_start), _ptr(base_pos), rows, B,
                                           H, T, D, _ptr(k_codes), _ptr(k_sz), _ptr(v_codes), _ptr(v_sz),
                                           _ptr(dev_status), _stream(stream))


def qspec_kv4_load(k_codes, k_sz, v_codes, v_sz, row_start, base_pos, rows, B, H, T, D, k, ldk, v, ldv,
                   dev_status=None, stream=None):
    return load_library().qspec_kv4_load(_ptr(k_codes), _ptr(k_sz), _ptr(v_codes), _ptr(v_sz), _ptr(row_start),
                                         _ptr(base_pos), rows, B, H, T, D, _ptr(k), ldk, _ptr(v), ldv,
                                         _ptr(dev_status), _stream(stream))


def qspec_attn_kv4_workspace_bytes(B, R, Hq, H, D):
    return int(load_library().qspec_attn_kv4_workspace_bytes(B, R, Hq, H, D))


def qspec_attn_kv4(q, ldq, k_codes, k_sz, v_codes, v_sz, length, B, R, Hq, H, T, D, scale, o, ldo, workspace,
                   ws_bytes, dev_status=None, stream=None):
    return load_library().qspec_attn_kv4(_ptr(q), ldq, _ptr(k_codes), _ptr(k_sz), _ptr(v_codes), _ptr(v_sz),
                                         _ptr(length), B, R, Hq, H, T, D, scale, _ptr(o), ldo, _ptr(workspace),
                                         ws_bytes, _ptr(dev_status), _stream(stream))


def qspec_attn_prompt(q, ldq, k, ldk, v, ldv, q_start, k_start, q_rows, k_rows, B, Hq, H, D, scale, o, ldo,
                      dev_status=None, stream=None):
    return load_library().qspec_attn_prompt(_ptr(q), ldq, _ptr(k), ldk, _ptr(v), ldv, _ptr(q_start),
                                            _ptr(k_start), q_rows, k_rows, B, Hq, H, D, scale, _ptr(o), ldo,
                                            _ptr(dev_status), _stream(stream))


def qspec_debug_attn_kv4_bounded(q, ldq, k_codes, k_sz, v_codes, v_sz, length, B, R, Hq, H, T, D, scale, o, ldo,
                                 workspace, ws_bytes, wait_limit, stall, dev_status=None, stream=None):
    return load_library().qspec_debug_attn_kv4_bounded(
        _ptr(q), ldq, _ptr(k_codes), _ptr(k_sz), _ptr(v_codes), _ptr(v_sz), _ptr(length), B, R, Hq, H, T, D, scale,
        _ptr(o), ldo, _ptr(workspace), ws_bytes, wait_limit, stall, _ptr(dev_status), _stream(stream))


def qspec_debug_attn_prompt_bounded(q, ldq, k, ldk, v, ldv, q_start, k_start, q_rows, k_rows, B, Hq, H, D, scale, o,
                                    ldo, wait_limit, stall, dev_status=None, stream=None):
    return load_library().qspec_debug_attn_prompt_bounded(
        _ptr(q), ldq, _ptr(k), ldk, _ptr(v), ldv, _ptr(q_start), _ptr(k_start), q_rows, k_rows, B, Hq, H, D, scale,
        _ptr(o), ldo, wait_limit, stall, _ptr(dev_status), _stream(stream))


# ---------------------------------------------------------------------------
# allocating conveniences (torch tensors in, torch tensors out)
# ---------------------------------------------------------------------------
@_allocates
def pack_weights(codes, s, z, dev_status=None, stream=None):
    """codes uint8 [N][K], s / z fp16 [N][K/128] -> (packed uint8 [N][K/2], sz int32 [N][K/128])."""
    _need(codes, torch.uint8, "codes")
    _need(s, torch.float16, "s")
    _need(z, torch.float16, "z")
    N, K = codes.shape
    packed = torch.empty((N, K // 2), dtype=torch.uint8, device=codes.device)
    sz = torch.empty((N, K // GROUP), dtype=torch.int32, device=codes.device)
    _check(qspec_pack_weights(codes, s, z, N, K, packed, sz, dev_status, stream),
           "qspec_pack_weights")
    return packed, sz


@_allocates
def quant_act_int4(x, dev_status=None, stream=None):
    """x bf16 [M][K] -> (xq uint8 [M][K/2], sx fp32 [M][G], qs int32 [M][G])."""
    _need(x, torch.bfloat16, "x")
    M, K = x.shape
    xq = torch.empty((M, K // 2), dtype=torch.uint8, device=x.device)
    sx = torch.empty((M, K // GROUP), dtype=torch.float32, device=x.device)
    qs = torch.empty((M, K // GROUP), dtype=torch.int32, device=x.device)
    _check(qspec_quant_act_int4(x, M, K, K, xq, sx, qs, dev_status, stream), "qspec_quant_act_int4")
    return xq, sx, qs


@_allocates
def linear_w4a4(xq, sx, qs, packed, sz, want_I=False, out=None, dev_status=None, stream=None):
    M, N, K = xq.shape[0], packed.shape[0], packed.shape[1] * 2
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    I = (torch.empty((M, N, K // GROUP), dtype=torch.int32, device=xq.device) if want_I else None)
    _check(qspec_linear_w4a4(xq, sx, qs, packed, sz, M, N, K, y, y.stride(0), I, dev_status,
                             stream), "qspec_linear_w4a4")
    return (y, I) if want_I else y


@_allocates
def linear_w4a4_bf16(x, packed, sz, want_I=False, out=None, dev_status=None, stream=None):
    """Quantise bf16 activations and run the W4A4 linear in one call:
    returns (y, xq, sx, qs) (and I when want_I), equal to quant_act_int4
    followed by linear_w4a4."""
    _need(x, torch.bfloat16, "x")
    M, K = x.shape
    N = packed.shape[0]
    dev = x.device
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    xq = torch.empty((M, K // 2), dtype=torch.uint8, device=dev)
    sx = torch.empty((M, K // GROUP), dtype=torch.float32, device=dev)
    qs = torch.empty((M, K // GROUP), dtype=torch.int32, device=dev)
    I = torch.empty((M, N, K // GROUP), dtype=torch.int32, device=dev) if want_I else None
    _check(qspec_linear_w4a4_bf16(x, x.stride(0), packed, sz, M, N, K, y, y.stride(0), xq, sx, qs, I,
                                  dev_status, stream), "qspec_linear_w4a4_bf16")
    return (y, xq, sx, qs, I) if want_I else (y, xq, sx, qs)


@_allocates
def linear_w4a16(x, packed, sz, out=None, dev_status=None, stream=None):
    _need(x, torch.bfloat16, "x")
    M, K = x.shape
    N = packed.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=x.device)
    _check(qspec_linear_w4a16(x, x.stride(0), packed, sz, M, N, K, y, y.stride(0), dev_status,
                              stream), "qspec_linear_w4a16")
    return y


def verify_workspace(B, gamma, V, device="cuda"):
    n = qspec_verify_workspace_bytes(B, gamma, V)
    if n == 0:
        raise QspecError(ERR_SHAPE, "qspec_verify_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


@_allocates
def verify_greedy(p, draft, workspace=None, dev_status=None, stream=None):
    B, g1, V = p.shape
    gamma = g1 - 1
    ws = workspace if workspace is not None else verify_workspace(B, gamma, V, p.device)
    n_acc = torch.empty(B, dtype=torch.int32, device=p.device)
    out = torch.empty((B, gamma + 1), dtype=torch.int32, device=p.device)
    _check(qspec_verify_greedy(p, draft, B, gamma, V, n_acc, out, ws, ws.numel(), dev_status,
                               stream), "qspec_verify_greedy")
    return n_acc, out


@_allocates
def verify_sample(p, q, draft, seed, rnd, workspace=None, dev_status=None, stream=None):
    B, g1, V = p.shape
    gamma = g1 - 1
    ws = workspace if workspace is not None else verify_workspace(B, gamma, V, p.device)
    n_acc = torch.empty(B, dtype=torch.int32, device=p.device)
    out = torch.empty((B, gamma + 1), dtype=torch.int32, device=p.device)
    _check(qspec_verify_sample(p, q, draft, B, gamma, V, seed, rnd, n_acc, out, ws, ws.numel(),
                               dev_status, stream), "qspec_verify_sample")
    return n_acc, out


def draft_workspace(B, V, device="cuda"):
    n = qspec_draft_workspace_bytes(B, V)
    if n == 0:
        raise QspecError(ERR_SHAPE, "qspec_draft_workspace_bytes")
    return torch.empty(n, dtype=torch.uint8, device=device)


@_allocates
def draft_sample(q, seed, rnd, step, workspace=None, dev_status=None, stream=None):
    """q bf16 [B][V] draft logits of draft position step (1..16) ->
    (token int32 [B], confidence fp32 [B], entropy fp32 [B])."""
    _need(q, torch.bfloat16, "q")
    B, V = q.shape
    ws = workspace if workspace is not None else draft_workspace(B, V, q.device)
    token = torch.empty(B, dtype=torch.int32, device=q.device)
    conf = torch.empty(B, dtype=torch.float32, device=q.device)
    ent = torch.empty(B, dtype=torch.float32, device=q.device)
    _check(qspec_draft_sample(q, B, V, seed, rnd, step, token, conf, ent, ws, ws.numel(), dev_status,
                              stream), "qspec_draft_sample")
    return token, conf, ent


def kv_overwrite(k_cache, v_cache, k_new, v_new, base_pos, n_acc, dev_status=None, stream=None):
    L, B, H, T, D = k_cache.shape
    gamma = k_new.shape[2] - 1
    _check(qspec_kv_overwrite(k_cache, v_cache, k_new, v_new, base_pos, n_acc, L, B, H, T, D,
                              gamma, dev_status, stream), "qspec_kv_overwrite")


@_allocates
def quant_weights_fp8(w16, dev_status=None, stream=None):
    """Parent weights fp16 [N][K] -> (w8 uint8 [N][K] E4M3, s8 fp32 [N])."""
    _need(w16, torch.float16, "w16")
    N, K = w16.shape
    w8 = torch.empty((N, K), dtype=torch.uint8, device=w16.device)
    s8 = torch.empty(N, dtype=torch.float32, device=w16.device)
    _check(qspec_quant_weights_fp8(w16, N, K, w8, s8, dev_status, stream), "qspec_quant_weights_fp8")
    return w8, s8


@_allocates
def quant_act_fp8(x, dev_status=None, stream=None):
    """bf16 [M][K] -> (xq uint8 [M][K] E4M3, sa fp32 [M])."""
    _need(x, torch.bfloat16, "x")
    M, K = x.shape
    xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    sa = torch.empty(M, dtype=torch.float32, device=x.device)
    _check(qspec_quant_act_fp8(x, M, K, x.stride(0), xq, sa, dev_status, stream), "qspec_quant_act_fp8")
    return xq, sa


@_allocates
def linear_fp8(xq, sa, w8, s8, out=None, dev_status=None, stream=None):
    M, K = xq.shape
    N = w8.shape[0]
    y = out if out is not None else torch.empty((M, N), dtype=torch.bfloat16, device=xq.device)
    _check(qspec_linear_fp8(xq, sa, w8, s8, M, N, K, y, y.stride(0), dev_status, stream), "qspec_linear_fp8")
    return y


def _heads(t, name):
    """A [rows][heads][D] bf16 CUDA tensor whose heads of a row are contiguous
    (rows may be strided, as columns of a fused projection's output are):
    (rows, heads, D, leading dimension)."""
    if t.device.type != "cuda" or t.dtype != torch.bfloat16 or t.dim() != 3:
        raise ValueError("%s must be a bf16 CUDA tensor [rows][heads][D]" % name)
    rows, H, D = t.shape
    if rows and (t.stride(2) != 1 or (H > 1 and t.stride(1) != D)):
        raise ValueError("%s: the heads of a row must be contiguous" % name)
    return rows, H, D, (t.stride(0) if rows > 1 else H * D)


@_allocates
def rmsnorm_fp8(x, w, eps, residual=None, want_bf16=False, dev_status=None, stream=None):
    """x bf16 [M][K] (plus residual bf16 [M][K]) -> (xq uint8 [M][K] E4M3, sa fp32 [M], h bf16 [M][K] or
    None without a residual, y bf16 [M][K] or None without want_bf16)."""
    _need(w, torch.bfloat16, "w")
    for t, name in ((x, "x"), (residual, "residual")):
        if t is not None and (t.device.type != "cuda" or t.dtype != torch.bfloat16 or t.dim() != 2
                              or t.shape != x.shape or (t.numel() and t.stride(1) != 1)):
            raise ValueError("%s must be a bf16 CUDA tensor [M][K] with contiguous rows" % name)
    M, K = x.shape
    if w.numel() != K:
        raise ValueError("w must hold %d values" % K)
    ld = lambda t: t.stride(0) if M > 1 else K      # noqa: E731
    xq = torch.empty((M, K), dtype=torch.uint8, device=x.device)
    sa = torch.empty(M, dtype=torch.float32, device=x.device)
    h = torch.empty((M, K), dtype=torch.bfloat16, device=x.device) if residual is not None else None
    y = torch.empty((M, K), dtype=torch.bfloat16, device=x.device) if want_bf16 else None
    _check(qspec_rmsnorm_fp8(x, ld(x), residual, K if residual is None else ld(residual), w, eps, M, K, h, K, xq,
                             sa, y, K, dev_status, stream), "qspec_rmsnorm_fp8")
    return xq, sa, h, y


def kv4_cache(B, H, T, D, device="cuda"):
    """A zeroed 4-bit cache of one layer: (k_codes uint8 [B][H][T][D/2], k_sz int32 [B][H][T], v_codes, v_sz)."""
    codes = lambda: torch.zeros((B, H, T, D // 2), dtype=torch.uint8, device=device)   # noqa: E731
    words = lambda: torch.zeros((B, H, T), dtype=torch.int32, device=device)           # noqa: E731
    return codes(), words(), codes(), words()


def _cache_shape(cache):
    k_codes, k_sz, v_codes, v_sz = cache
    for t, dt, name in ((k_codes, torch.uint8, "k_codes"), (v_codes, torch.uint8, "v_codes"),
                        (k_sz, torch.int32, "k_sz"), (v_sz, torch.int32, "v_sz")):
        _need(t, dt, name)
    B, H, T, D2 = k_codes.shape
    if v_codes.shape != k_codes.shape or k_sz.shape != (B, H, T) or v_sz.shape != (B, H, T):
        raise ValueError("codes must be [B][H][T][D/2] and scale words [B][H][T], for K and V alike")
    return B, H, T, 2 * D2


def _starts(t, B, name):
    _need(t, torch.int32, name)
    if t.numel() != B:
        raise ValueError("%s must hold %d values" % (name, B))


def kv4_append(cache, k, v, row_start, base_pos, dev_status=None, stream=None):
    """Quantise packed rows k, v bf16 [rows][H][D] into a cache (as kv4_cache gives it): rows row_start[b] ..
    row_start[b + 1] - 1 become positions base_pos[b], base_pos[b] + 1, ... of sequence b."""
    B, H, T, D = _cache_shape(cache)
    rows, Hk, Dk, ldk = _heads(k, "k")
    rv, Hv, Dv, ldv = _heads(v, "v")
    if (Hk, Dk) != (H, D) or (rv, Hv, Dv) != (rows, H, D):
        raise ValueError("k and v must be [rows][%d][%d]" % (H, D))
    _starts(row_start, B + 1, "row_start")
    _starts(base_pos, B, "base_pos")
    k_codes, k_sz, v_codes, v_sz = cache
    _check(qspec_kv4_append(k, ldk, v, ldv, row_start, base_pos, rows, B, H, T, D, k_codes, k_sz, v_codes, v_sz,
                            dev_status, stream), "qspec_kv4_append")


@_allocates
def kv4_load(cache, row_start, base_pos, rows, dev_status=None, stream=None):
    """The rows of kv4_append back from the cache: (k, v) bf16 [rows][H][D].  Rows of no sequence are zeros."""
    B, H, T, D = _cache_shape(cache)
    _starts(row_start, B + 1, "row_start")
    _starts(base_pos, B, "base_pos")
    k_codes, k_sz, v_codes, v_sz = cache
    k = torch.zeros((rows, H, D), dtype=torch.bfloat16, device=k_codes.device)
    v = torch.zeros_like(k)
    _check(qspec_kv4_load(k_codes, k_sz, v_codes, v_sz, row_start, base_pos, rows, B, H, T, D, k, H * D, v, H * D,
                          dev_status, stream), "qspec_kv4_load")
    return k, v


def attn_kv4_workspace(B, R, Hq, H, D, device="cuda"):
    """Workspace of attn_kv4, zeroed as its first use needs it."""
    n = qspec_attn_kv4_workspace_bytes(B, R, Hq, H, D)
    if n == 0:
        raise QspecError(ERR_SHAPE, "qspec_attn_kv4_workspace_bytes")
    return torch.zeros(n, dtype=torch.uint8, device=device)


@_allocates
def attn_kv4(q, cache, length, scale, workspace=None, out=None, dev_status=None, stream=None):
    """q bf16 [B R][Hq][D], the newest R rows of each sequence, over a 4-bit cache; length int32 [B] counts them.
    Returns o bf16 [B R][Hq][D]."""
    B, H, T, D = _cache_shape(cache)
    rows, Hq, Dq, ldq = _heads(q, "q")
    if Dq != D or rows % B:
        raise ValueError("q must be [B R][Hq][%d] with B = %d" % (D, B))
    _starts(length, B, "length")
    R = rows // B
    o = out if out is not None else torch.empty((rows, Hq, D), dtype=torch.bfloat16, device=q.device)
    if _heads(o, "out")[:3] != (rows, Hq, D):
        raise ValueError("out must be [%d][%d][%d]" % (rows, Hq, D))
    if workspace is None:
        workspace = attn_kv4_workspace(B, R, Hq, H, D, q.device)
    k_codes, k_sz, v_codes, v_sz = cache
    _check(qspec_attn_kv4(q, ldq, k_codes, k_sz, v_codes, v_sz, length, B, R, Hq, H, T, D, scale, o,
                          _heads(o, "out")[3], workspace, workspace.numel(), dev_status, stream), "qspec_attn_kv4")
    return o


@_allocates
def attn_prompt(q, k, v, q_start, k_start=None, scale=None, out=None, dev_status=None, stream=None):
    """Causal attention over packed prompts: q bf16 [q_rows][Hq][D], k and v bf16 [k_rows][H][D], q_start and
    k_start int32 [B + 1] (k_start None: the same).  scale None: 1 / sqrt(D).  Returns o bf16 [q_rows][Hq][D]."""
    q_rows, Hq, D, ldq = _heads(q, "q")
    k_rows, H, Dk, ldk = _heads(k, "k")
    rv, Hv, Dv, ldv = _heads(v, "v")
    if Dk != D or (rv, Hv, Dv) != (k_rows, H, D):
        raise ValueError("k and v must be [k_rows][H][%d]" % D)
    k_start = q_start if k_start is None else k_start
    B = q_start.numel() - 1
    _starts(q_start, B + 1, "q_start")
    _starts(k_start, B + 1, "k_start")
    o = out if out is not None else torch.empty((q_rows, Hq, D), dtype=torch.bfloat16, device=q.device)
    if _heads(o, "out")[:3] != (q_rows, Hq, D):
        raise ValueError("out must be [%d][%d][%d]" % (q_rows, Hq, D))
    _check(qspec_attn_prompt(q, ldq, k, ldk, v, ldv, q_start, k_start, q_rows, k_rows, B, Hq, H, D,
                             D ** -0.5 if scale is None else scale, o, _heads(o, "out")[3], dev_status, stream),
           "qspec_attn_prompt")
    return o
