// fp8_block.cuh -- what the products of E4M3 codes with a scale for each block
// of 128 share: their arguments, the gated one's function, and the ends of sums that
// lie in shared memory.
#pragma once

#include <cuda_fp8.h>

#include "qspec_device.cuh"
#include "umma.cuh"

namespace qspec {
namespace f8b {

constexpr int kMaxM = 1 << 22, kMaxN = 1 << 30;   // what the grids count

struct Args {
    const float *sa;             // [K / 128][lds] scales of the tokens
    const float *s0, *s1;        // [ceil(N / 128)][K / 128] scales of the weights (gated: gate, up)
    uint16_t *y;                 // bf16 output (gated: may be null)
    uint8_t *hq;                 // gated: E4M3 output and its scales [N / 128][ldh] (may be null)
    float *sh;
    int32_t *st;
    int lds, M, N, K, ldy, ldh;
};

// two fp32 values in a register pair, and packed operations on them
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float lo32(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi32(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t add2(uint64_t a, uint64_t b) {
    uint64_t d;
    asm("add.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(a), "l"(b));
    return d;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
// max(a, |b|, |c|) and max(a, b) that keep a NaN (a >= 0)
__device__ __forceinline__ float max_abs(float a, float b, float c) {
    float d;
    asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ float max_nan(float a, float b) {
    float d;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
    return d;
}

// shared-memory descriptor of a K-major operand with rows of 128 bytes in the 128-byte swizzle (fp8.cu)
__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

// h = silu(g) u = g u / (1 + exp(-g)).  exp(-g) passes fp32 below -88.7: 1 / inf is the limit 0; a NaN stays one.
__device__ __forceinline__ float gated(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// amax / 448: the quotient's two steps (fp8_block.cu) with 1 / 448 rounded; the division at fp32's ends.
__device__ __forceinline__ float scale_of(float amax) {
    constexpr float kY = 1.0f / 448.0f;
    if (!(amax > 1.0e-30f && amax < 1.0e38f)) return __fdiv_rn(amax, 448.0f);
    const float q = __fmul_rn(amax, kY);
    return __fmaf_rn(__fmaf_rn(-q, 448.0f, amax), kY, q);
}
// 1 / s by one Newton step, for s within 2^-126 .. 2^126.
__device__ __forceinline__ float reciprocal(float s) {
    const float y = rcp_approx(s);
    return __fmaf_rn(__fmaf_rn(-s, y, 1.0f), y, y);
}

constexpr float kSubnormal = 0x1.cp-118f, kNothing = 0x1.cp-142f;       // 448 x 2^-126, 2^-150: maxima below the one have a subnormal scale, up to the other one of 0

// A power of two that brings a maximum to where its reciprocal is a normal number: 2^96, 2^-96 or 1.
__device__ __forceinline__ float lift(float top) {
    return top < 1.0e-30f ? 7.9228162514264338e28f : top > 1.0e30f ? 1.262177448353619e-29f : 1.0f;
}

// A block's scale and what its codes are taken with: E4M3(v up inv), inv = 448 / (up max |v|), up a power of two that
// keeps the reciprocal inside fp32.  Within 3 x 2^-24 of v / s in the quotient.  A scale of 0 has the codes 0.
struct Quant {
    float s, inv, up;
    __device__ __forceinline__ explicit Quant(float amax) {
        if (amax < kSubnormal) amax = 448.0f * scale_of(amax);                      // (the scale as it is stored)
        up = lift(amax);
        s = scale_of(amax);
        inv = s > 0.0f ? 448.0f * reciprocal(amax * up) : 0.0f;
    }
};

// 32 neighbouring bytes (`wide`: on a multiple of 32, else of 16)
__device__ __forceinline__ void store32(void *p, const uint32_t (&w)[8], bool wide) {
    if (wide) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};\n" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        reinterpret_cast<uint4 *>(p)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4 *>(p)[1] = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// four codes, the first in the low byte
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

// Four neighbouring channels n .. n + 3 of token m in bf16.
__device__ __forceinline__ void store_bf16(const Args &a, int m, int n, const float (&v)[4]) {
    uint16_t *y = a.y + (size_t)m * a.ldy + n;
    if ((reinterpret_cast<uintptr_t>(y) & 7) == 0 && n + 4 <= a.N) {
        *reinterpret_cast<uint2 *>(y) =
            make_uint2((uint32_t)float_to_bf16_bits(v[0]) | (uint32_t)float_to_bf16_bits(v[1]) << 16,
                       (uint32_t)float_to_bf16_bits(v[2]) | (uint32_t)float_to_bf16_bits(v[3]) << 16);
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e)
            if (n + e < a.N) y[e] = float_to_bf16_bits(v[e]);
    }
}

// The gated product's outputs for token m and the 128 channels of block `block` by a warp, four channels to a lane.
__device__ __forceinline__ void store_gated(const Args &a, int m, int block, int lane, const float (&g)[4], const float (&u)[4]) {
    float h[4], amax = 0.0f;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        h[e] = gated(g[e], u[e]);
        amax = max_nan(amax, fabsf(h[e]));
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if (a.hq != nullptr) {
        const Quant q(amax);
        reinterpret_cast<uint32_t *>(a.hq + (size_t)m * a.N + (size_t)block * kGroup)[lane] =
            q.s == 0.0f ? 0u : codes4(h[0] * q.up * q.inv, h[1] * q.up * q.inv, h[2] * q.up * q.inv, h[3] * q.up * q.inv);
        if (lane == 0) a.sh[(size_t)block * a.ldh + m] = q.s;
    }
    if (lane == 0 && !(amax < (a.y != nullptr ? 3.3961775292304601e38f : INFINITY))) flag(a.st, QSPEC_ERR_NONFINITE);
    if (a.y != nullptr) store_bf16(a, m, block * kGroup + 4 * lane, h);
}

// Sums over a cluster's parts of K, in their order: four floats at each of `at` in the shared memory of the CTAs first ..
// first + split - 1 (R of them at most).  All are asked for before the first is added: an answer takes about a
// microsecond.
constexpr int kMaxSplit = 8;
template <int R = kMaxSplit, int T>
__device__ __forceinline__ void sum_parts(const float *const (&at)[T], int split, int first, float (&v)[T][4]) {
    uint4 w[T][R];
#pragma unroll
    for (int t = 0; t < T; ++t)
#pragma unroll
        for (int r = 0; r < R; ++r)
            w[t][r] = r < split ? umma::ld_peer_v4(at[t], (uint32_t)(first + r)) : make_uint4(0, 0, 0, 0);
#pragma unroll
    for (int t = 0; t < T; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) v[t][e] = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
            v[t][0] += __uint_as_float(w[t][r].x);
            v[t][1] += __uint_as_float(w[t][r].y);
            v[t][2] += __uint_as_float(w[t][r].z);
            v[t][3] += __uint_as_float(w[t][r].w);
        }
    }
}

}  // namespace f8b
}  // namespace qspec
