// fp8_block.cu -- E4M3 codes with a scale for each block of 128: the quantisers
// of weights (128 x 128) and of activations (one token x 128).
//
//   s = amax / 448 (fp32, IEEE division), code = E4M3(v / s) (fp32 IEEE
//   quotient, round to nearest even, saturated at 448); a block of zeros has
//   s = 0 and codes 0.
//
// The quotient takes two fused steps from the correctly rounded reciprocal y of
// s: q = v y, t = q + y (v - q s), the remainder exact.  That is the IEEE quotient
// wherever nothing under- or overflows on the way (Markstein, "Computation of
// elementary functions on the IBM RISC System/6000 processor", IBM J. Res.
// Dev. 34, 1990).  Scales outside (2^-80, 2^80) take the division; inside, a value
// with a code that is not 0 is at least 2^-90, and its remainder's last place, 47
// below its first, is a number.
//
// Bound: HBM (2 bytes in, 1 out per value).  Half a warp has one token's 128
// values, 16 bytes to a lane; a CTA takes 4 neighbouring blocks of up to 32
// tokens, so that reads are 1 KB at a time and the scales, which lie token by
// token, go out 128 bytes at a time through shared memory.
#include <climits>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "qspec_device.cuh"
#include "qspec_host.h"

namespace qspec {

namespace {

namespace f8b {

constexpr int kThreads = 256;
constexpr int kHalves = kThreads / 16;          // half warps
constexpr int kBlocksX = 4;                     // neighbouring blocks per CTA

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
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}

// a word of two fp16 or bf16 values
template <bool kHalf>
__device__ __forceinline__ uint64_t both(uint32_t w) {
    if constexpr (kHalf) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        return f2(f.x, f.y);
    }
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
template <bool kHalf>
__device__ __forceinline__ float max_of(uint4 v, float amax) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        const uint64_t f = both<kHalf>(w[e]);
        amax = max_abs(amax, lo32(f), hi32(f));
    }
    return amax;
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {          // the first in the low byte
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// the codes of 8 values over the scale s; one of 0 stands for a block of zeros
template <bool kHalf>
__device__ __forceinline__ uint2 codes_of(uint4 v, float s, float y) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t c[4];
    if (s > 8.271806125530277e-25f && s < 1.2089258196146292e24f) {        // 2^-80, 2^80
        const uint64_t yy = f2(y, y), ss = f2(-s, -s);
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t f = both<kHalf>(w[e]), q = mul2(f, yy), t = fma2(fma2(q, ss, f), yy, q);
            c[e] = pack_e4m3(copysignf(lo32(t), lo32(f)), copysignf(hi32(t), hi32(f)));      // (-0 stays -0)
        }
    } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t f = both<kHalf>(w[e]);
            c[e] = s == 0.0f ? 0u : pack_e4m3(__fdiv_rn(lo32(f), s), __fdiv_rn(hi32(f), s));
        }
    }
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// NI items (token, block) per half warp: NI * kHalves / kBlocksX tokens per CTA
template <int NI>
__global__ void __launch_bounds__(kThreads)
    quant_act_kernel(const uint16_t *__restrict__ x, int M, int K, int ldx, uint8_t *__restrict__ xq,
                     float *__restrict__ sa, int lds, int32_t *st) {
    constexpr int kRows = NI * kHalves / kBlocksX;
    __shared__ float scales[kBlocksX][kRows];
    const int half = threadIdx.x >> 4, lane = threadIdx.x & 15;
    const int G = K / kGroup, across = (G + kBlocksX - 1) / kBlocksX;
    const int g0 = (int)(blockIdx.x % (unsigned)across) * kBlocksX, r0 = (int)(blockIdx.x / (unsigned)across) * kRows;
    const int g = g0 + half % kBlocksX;
    pdl_launch_dependents();
    pdl_wait();
    uint4 v[NI];
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int m = r0 + half / kBlocksX + i * (kHalves / kBlocksX);
        v[i] = m < M && g < G ? __ldcs(reinterpret_cast<const uint4 *>(x + (size_t)m * ldx + (size_t)g * kGroup) + lane)
                              : make_uint4(0, 0, 0, 0);
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < NI; ++i) {
        const int r = half / kBlocksX + i * (kHalves / kBlocksX), m = r0 + r;
        float amax = max_of<false>(v[i], 0.0f);
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float s = __fdiv_rn(amax, 448.0f);
        bad |= !(amax < INFINITY);
        const uint2 c = codes_of<false>(v[i], s, __frcp_rn(s));
        if (m < M && g < G) reinterpret_cast<uint2 *>(xq + (size_t)m * K + (size_t)g * kGroup)[lane] = c;
        if (lane == 0) scales[half % kBlocksX][r] = s;
    }
    const int bad_any = __syncthreads_or(bad ? 1 : 0);
    for (int i = threadIdx.x; i < kBlocksX * kRows; i += kThreads) {
        const int gg = g0 + i / kRows, m = r0 + i % kRows;
        if (gg < G && m < M) sa[(size_t)gg * lds + m] = scales[i / kRows][i % kRows];
    }
    if (threadIdx.x == 0 && bad_any) flag(st, QSPEC_ERR_NONFINITE);
}

// one 128 x 128 block per CTA, kept in registers between its load and its codes
__global__ void __launch_bounds__(kThreads, 3)
    quant_weights_kernel(const uint16_t *__restrict__ w, int N, int K, uint8_t *__restrict__ w8, float *__restrict__ sw,
                         int32_t *st) {
    constexpr int kPer = kGroup / kHalves;       // rows per half warp
    __shared__ float red[kThreads / 32];
    const int half = threadIdx.x >> 4, lane = threadIdx.x & 15, warp = threadIdx.x >> 5;
    const int G = K / kGroup, g = (int)(blockIdx.x % (unsigned)G), nb = (int)(blockIdx.x / (unsigned)G), n0 = nb * kGroup;
    pdl_wait();
    uint4 v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int n = n0 + half + i * kHalves;
        v[i] = n < N ? __ldcs(reinterpret_cast<const uint4 *>(w + (size_t)n * K + (size_t)g * kGroup) + lane)
                     : make_uint4(0, 0, 0, 0);
    }
    float amax = 0.0f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) amax = max_of<true>(v[i], amax);
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    if ((threadIdx.x & 31) == 0) red[warp] = amax;
    __syncthreads();
    amax = red[0];
#pragma unroll
    for (int i = 1; i < kThreads / 32; ++i) amax = max_nan(amax, red[i]);
    const float s = __fdiv_rn(amax, 448.0f), y = __frcp_rn(s);
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        const int n = n0 + half + i * kHalves;
        const uint2 c = codes_of<true>(v[i], s, y);
        if (n < N) reinterpret_cast<uint2 *>(w8 + (size_t)n * K + (size_t)g * kGroup)[lane] = c;
    }
    if (threadIdx.x == 0) {
        sw[(size_t)nb * G + g] = s;
        if (!(amax < INFINITY)) flag(st, QSPEC_ERR_NONFINITE);
    }
    // Only now may the next kernel begin: a product behind this one reads its weights ahead of its dependency wait.  (A
    // CTA's first thread to come here speaks for all of them.)
    __threadfence();
    __syncthreads();
    pdl_launch_dependents();
}

template <int NI>
int launch_act(const uint16_t *x, int M, int K, int ldx, uint8_t *xq, float *sa, int lds, int32_t *st, cudaStream_t s) {
    constexpr int kRows = NI * kHalves / kBlocksX;
    const long long ctas = (long long)((K / kGroup + kBlocksX - 1) / kBlocksX) * (((long long)M + kRows - 1) / kRows);
    return launch_pdl("qspec_quant_act_fp8_block", quant_act_kernel<NI>, dim3((unsigned)ctas), dim3(kThreads), 0, s, x, M, K, ldx, xq, sa, lds, st);
}

}  // namespace f8b

}  // namespace

}  // namespace qspec

using namespace qspec;

extern "C" int qspec_quant_weights_fp8_block(const uint16_t *w_fp16, int N, int K, uint8_t *w8, float *sw,
                                             int32_t *dev_status, qspec_stream_t stream) {
    if (!w_fp16 || !w8 || !sw) return QSPEC_ERR_NULL;
    if (N < 1 || K < kGroup || K % kGroup) return QSPEC_ERR_SHAPE;
    if (!aligned(w_fp16, 16) || !aligned(w8, 8) || !aligned(sw, 4)) return QSPEC_ERR_ALIGN;
    const long long blocks = (long long)(K / kGroup) * (((long long)N + kGroup - 1) / kGroup);
    if (blocks > INT_MAX) return QSPEC_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    return launch_pdl("qspec_quant_weights_fp8_block", f8b::quant_weights_kernel, dim3((unsigned)blocks), dim3(f8b::kThreads), 0,
                      as_cuda(stream), w_fp16, N, K, w8, sw, dev_status);
}

extern "C" int qspec_quant_act_fp8_block(const uint16_t *x_bf16, int M, int K, int ldx, uint8_t *xq, float *sa, int lds,
                                         int32_t *dev_status, qspec_stream_t stream) {
    if (!x_bf16 || !xq || !sa) return QSPEC_ERR_NULL;
    if (M < 1 || K < kGroup || K % kGroup || ldx < K || lds < M || (long long)(K / kGroup) * M > INT_MAX) return QSPEC_ERR_SHAPE;
    if (!aligned(x_bf16, 16) || ldx % 8 || !aligned(xq, 8) || !aligned(sa, 4)) return QSPEC_ERR_ALIGN;
    int rc = check_device();
    if (rc) return rc;
    cudaStream_t s = as_cuda(stream);
    if ((long long)M * K < 1 << 22) return f8b::launch_act<2>(x_bf16, M, K, ldx, xq, sa, lds, dev_status, s);
    return f8b::launch_act<8>(x_bf16, M, K, ldx, xq, sa, lds, dev_status, s);
}
