// fp8_block.cu -- E4M3 codes with a scale for each block of 128: the quantisers
// of weights (128 x 128) and of activations (one token x 128).
//
//   s = amax / 448 (fp32, IEEE division), code = E4M3(v / s) (fp32 IEEE
//   quotient, round to nearest even, saturated at 448); a block of zeros has
//   s = 0 and codes 0.
//
// The quotient takes two fused steps from the reciprocal y of s: q = v y, t = q + y (v - q s),
// the remainder exact.  With y correctly rounded that is the IEEE quotient wherever nothing
// under- or overflows on the way (Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", IBM J. Res. Dev. 34, 1990); y here is one Newton step from the
// approximate reciprocal, in the last place the correctly rounded one or its neighbour, and
// the codes are the division's for all values of either type over the scales of all maxima
// (tests/test_gpu_fp8_block.py goes through them).  Scales outside (2^-80, 2^80) take
// the division; inside, a value with a code that is not 0 is at least 2^-90, and its
// remainder's last place, 47 below its first, is a number.
//
// Bound: HBM (2 bytes in, 1 out per value).  8 lanes have one token's 128 values, 32 bytes
// to a lane (16 lanes and 16 bytes where addresses are no multiples of 32: 4099 x 14336 in
// 29.9 us for 28.0, 6.4 TB/s, with seven CTAs to an SM and 36 bytes of spills); a CTA takes 4 neighbouring blocks of some tokens, so that reads are
// 1 KB at a time and the scales, which lie token by token, go out in runs through
// shared memory.  With the divisions of s and y, 16 lanes and half the CTAs resident
// it took 34.7 us.
#include <algorithm>
#include <climits>

#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "fp8_block.cuh"
#include "qspec_host.h"

namespace qspec {

namespace {

namespace f8q {

using f8b::f2;
using f8b::fma2;
using f8b::hi32;
using f8b::lo32;
using f8b::max_abs;
using f8b::max_nan;
using f8b::mul2;

constexpr int kThreads = 256;
constexpr int kBlocksX = 4;                     // neighbouring blocks per CTA

// a word of two fp16 or bf16 values
template <bool kHalf>
__device__ __forceinline__ uint64_t both(uint32_t w) {
    if constexpr (kHalf) {
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w));
        return f2(f.x, f.y);
    }
    return f2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
// W words of a row; 8 of them, 32 bytes, in one load
template <int W>
struct Words {
    uint32_t w[W];
};
template <int W>
__device__ __forceinline__ Words<W> load(const uint16_t *p, bool in) {
    Words<W> v;
#pragma unroll
    for (int e = 0; e < W; ++e) v.w[e] = 0;
    if (in) {
        if constexpr (W == 8) {
            asm volatile("ld.global.cs.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];\n"
                         : "=r"(v.w[0]), "=r"(v.w[1]), "=r"(v.w[2]), "=r"(v.w[3]), "=r"(v.w[4]), "=r"(v.w[5]), "=r"(v.w[6]), "=r"(v.w[7])
                         : "l"(p));
        } else {
            const uint4 u = __ldcs(reinterpret_cast<const uint4 *>(p));
            v.w[0] = u.x, v.w[1] = u.y, v.w[2] = u.z, v.w[3] = u.w;
        }
    }
    return v;
}
template <bool kHalf, int W>
__device__ __forceinline__ float max_of(const Words<W> &v, float amax) {
#pragma unroll
    for (int e = 0; e < W; ++e) {
        const uint64_t f = both<kHalf>(v.w[e]);
        amax = max_abs(amax, lo32(f), hi32(f));
    }
    return amax;
}

__device__ __forceinline__ uint32_t pack_e4m3(float a, float b) {          // the first in the low byte
    return __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
}

// the codes of 2 W values over the scale s, stored; s = 0 stands for a block of zeros
template <bool kHalf, int W>
__device__ __forceinline__ void store_codes(uint8_t *out, const Words<W> &v, float s, float y, bool in) {
    uint32_t c[W / 2];
    if (s > 8.271806125530277e-25f && s < 1.2089258196146292e24f) {        // 2^-80, 2^80
        const uint64_t yy = f2(y, y), ss = f2(-s, -s);
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const uint64_t f = both<kHalf>(v.w[e]), q = mul2(f, yy), t = fma2(fma2(q, ss, f), yy, q);
            const uint32_t h = pack_e4m3(copysignf(lo32(t), lo32(f)), copysignf(hi32(t), hi32(f)));      // (-0 stays -0)
            c[e / 2] = e % 2 == 0 ? h : c[e / 2] | h << 16;
        }
    } else {
#pragma unroll
        for (int e = 0; e < W; ++e) {
            const uint64_t f = both<kHalf>(v.w[e]);
            const uint32_t h = s == 0.0f ? 0u : pack_e4m3(__fdiv_rn(lo32(f), s), __fdiv_rn(hi32(f), s));
            c[e / 2] = e % 2 == 0 ? h : c[e / 2] | h << 16;
        }
    }
    if (!in) return;
    if constexpr (W == 8)
        *reinterpret_cast<uint4 *>(out) = make_uint4(c[0], c[1], c[2], c[3]);
    else
        *reinterpret_cast<uint2 *>(out) = make_uint2(c[0], c[1]);
}

// teams of 64 / W lanes, each with NI items (token, block)
template <int W>
struct Act {
    static constexpr int kTeam = 64 / W, kTeams = kThreads / kTeam, kItems = W == 8 ? 2 : 4, kRows = kItems * kTeams / kBlocksX;
};

template <int W>
__global__ void __launch_bounds__(kThreads, (W == 8 ? 6 : 7))
    quant_act_kernel(const uint16_t *__restrict__ x, int M, int K, int ldx, uint8_t *__restrict__ xq,
                     float *__restrict__ sa, int lds, int32_t *st) {
    using A = Act<W>;
    __shared__ float scales[kBlocksX][A::kRows];
    const int team = threadIdx.x / A::kTeam, lane = threadIdx.x % A::kTeam;
    const int G = K / kGroup, across = (G + kBlocksX - 1) / kBlocksX;
    const int g0 = (int)(blockIdx.x % (unsigned)across) * kBlocksX, r0 = (int)(blockIdx.x / (unsigned)across) * A::kRows;
    const int g = g0 + team % kBlocksX;
    const size_t col = (size_t)g * kGroup + lane * 2 * W;
    pdl_launch_dependents();
    pdl_wait();
    Words<W> v[A::kItems];
#pragma unroll
    for (int i = 0; i < A::kItems; ++i) {
        const int m = r0 + team / kBlocksX + i * (A::kTeams / kBlocksX);
        v[i] = load<W>(x + (size_t)m * ldx + col, m < M && g < G);
    }
    bool bad = false;
#pragma unroll
    for (int i = 0; i < A::kItems; ++i) {
        const int r = team / kBlocksX + i * (A::kTeams / kBlocksX), m = r0 + r;
        float amax = max_of<false, W>(v[i], 0.0f);
#pragma unroll
        for (int o = A::kTeam / 2; o >= 1; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        const float s = f8b::scale_of(amax);
        bad |= !(amax < INFINITY);
        store_codes<false, W>(xq + (size_t)m * K + col, v[i], s, f8b::reciprocal(s), m < M && g < G);
        if (lane == 0) scales[team % kBlocksX][r] = s;
    }
    const int bad_any = __syncthreads_or(bad ? 1 : 0);
    for (int i = threadIdx.x; i < kBlocksX * A::kRows; i += kThreads) {
        const int gg = g0 + i / A::kRows, m = r0 + i % A::kRows;
        if (gg < G && m < M) sa[(size_t)gg * lds + m] = scales[i / A::kRows][i % A::kRows];
    }
    if (threadIdx.x == 0 && bad_any) flag(st, QSPEC_ERR_NONFINITE);
}

// One 128 x 128 block after another, kept in registers between its load and its codes, the next one's loads under way
// meanwhile: 3584 x 18944 in 32.9 us, 6.2 TB/s (35.7 with three CTAs to an SM and no loads ahead).
template <int W>
__global__ void __launch_bounds__(kThreads, 2)
    quant_weights_kernel(const uint16_t *__restrict__ w, int N, int K, int blocks, uint8_t *__restrict__ w8,
                         float *__restrict__ sw, int32_t *st) {
    constexpr int kTeam = 64 / W, kTeams = kThreads / kTeam, kPer = kGroup / kTeams;       // rows per team
    __shared__ float red[2][kThreads / 32];
    const int team = threadIdx.x / kTeam, lane = threadIdx.x % kTeam, warp = threadIdx.x >> 5;
    const int G = K / kGroup;
    pdl_wait();
    Words<W> v[2][kPer];
    auto fetch = [&](int b, Words<W> (&d)[kPer]) {
        const int nb = b / G, g = b - nb * G, n0 = nb * kGroup + team;
        const uint16_t *p = w + (size_t)n0 * K + (size_t)g * kGroup + lane * 2 * W;
#pragma unroll
        for (int i = 0; i < kPer; ++i) d[i] = load<W>(p + (size_t)(i * kTeams) * K, b < blocks && n0 + i * kTeams < N);
    };
    // a block's maximum, scale and codes
    auto code = [&](int b, const Words<W> (&d)[kPer], int turn) {
        const int nb = b / G, g = b - nb * G, n0 = nb * kGroup + team;
        uint8_t *p = w8 + (size_t)n0 * K + (size_t)g * kGroup + lane * 2 * W;
        float amax = 0.0f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) amax = max_of<true, W>(d[i], amax);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
        if ((threadIdx.x & 31) == 0) red[turn][warp] = amax;
        __syncthreads();
        amax = red[turn][0];
#pragma unroll
        for (int i = 1; i < kThreads / 32; ++i) amax = max_nan(amax, red[turn][i]);
        const float s = f8b::scale_of(amax), y = f8b::reciprocal(s);
#pragma unroll
        for (int i = 0; i < kPer; ++i) store_codes<true, W>(p + (size_t)(i * kTeams) * K, d[i], s, y, n0 + i * kTeams < N);
        if (threadIdx.x == 0) {
            sw[(size_t)nb * G + g] = s;
            if (!(amax < INFINITY)) flag(st, QSPEC_ERR_NONFINITE);
        }
    };
    int b = blockIdx.x;
    fetch(b, v[0]);
    for (; b < blocks; b += 2 * gridDim.x) {
        fetch(b + gridDim.x, v[1]);
        code(b, v[0], 0);
        if (b + (int)gridDim.x >= blocks) break;
        fetch(b + 2 * gridDim.x, v[0]);
        code(b + gridDim.x, v[1], 1);
    }
    // A product behind this kernel reads its weights ahead of its dependency wait, by asynchronous copies.  So the next
    // kernel begins only when this grid is complete (it never lets it begin earlier), each thread's codes performed for
    // the device and ordered before such copies.  (A fence behind every block took 3 us at 4099 x 14336.)
    __threadfence();
    umma::fence_proxy_async_global();
}

template <int W>
int launch_act(const uint16_t *x, int M, int K, int ldx, uint8_t *xq, float *sa, int lds, int32_t *st, cudaStream_t s) {
    const long long ctas = (long long)((K / kGroup + kBlocksX - 1) / kBlocksX) * (((long long)M + Act<W>::kRows - 1) / Act<W>::kRows);
    return launch_pdl("qspec_quant_act_fp8_block", quant_act_kernel<W>, dim3((unsigned)ctas), dim3(kThreads), 0, s, x, M, K, ldx, xq, sa, lds, st);
}

template <int W>
int launch_weights(const uint16_t *w, int N, int K, int blocks, uint8_t *w8, float *sw, int32_t *st, cudaStream_t s) {
    return launch_pdl("qspec_quant_weights_fp8_block", quant_weights_kernel<W>, dim3((unsigned)std::min(blocks, 2 * sm_count())),
                      dim3(kThreads), 0, s, w, N, K, blocks, w8, sw, st);
}

}  // namespace f8q

}  // namespace

}  // namespace qspec

using namespace qspec;

extern "C" int qspec_quant_weights_fp8_block(const uint16_t *w_fp16, int N, int K, uint8_t *w8, float *sw,
                                             int32_t *dev_status, qspec_stream_t stream) {
    if (!w_fp16 || !w8 || !sw) return QSPEC_ERR_NULL;
    if (N < 1 || K < kGroup || K % kGroup) return QSPEC_ERR_SHAPE;
    if (!aligned(w_fp16, 16) || !aligned(w8, 8) || !aligned(sw, 4)) return QSPEC_ERR_ALIGN;
    const long long blocks = (long long)(K / kGroup) * (((long long)N + kGroup - 1) / kGroup);
    if (blocks > INT_MAX / 2) return QSPEC_ERR_SHAPE;
    int rc = check_device();
    if (rc) return rc;
    cudaStream_t s = as_cuda(stream);
    // 32 bytes to a lane where the addresses allow it
    if (aligned(w_fp16, 32) && aligned(w8, 16)) return f8q::launch_weights<8>(w_fp16, N, K, (int)blocks, w8, sw, dev_status, s);
    return f8q::launch_weights<4>(w_fp16, N, K, (int)blocks, w8, sw, dev_status, s);
}

extern "C" int qspec_quant_act_fp8_block(const uint16_t *x_bf16, int M, int K, int ldx, uint8_t *xq, float *sa, int lds,
                                         int32_t *dev_status, qspec_stream_t stream) {
    if (!x_bf16 || !xq || !sa) return QSPEC_ERR_NULL;
    if (M < 1 || K < kGroup || K % kGroup || ldx < K || lds < M || (long long)(K / kGroup) * M > INT_MAX) return QSPEC_ERR_SHAPE;
    if (!aligned(x_bf16, 16) || ldx % 8 || !aligned(xq, 8) || !aligned(sa, 4)) return QSPEC_ERR_ALIGN;
    int rc = check_device();
    if (rc) return rc;
    cudaStream_t s = as_cuda(stream);
    if (aligned(x_bf16, 32) && ldx % 16 == 0 && aligned(xq, 16))
        return f8q::launch_act<8>(x_bf16, M, K, ldx, xq, sa, lds, dev_status, s);
    return f8q::launch_act<4>(x_bf16, M, K, ldx, xq, sa, lds, dev_status, s);
}
