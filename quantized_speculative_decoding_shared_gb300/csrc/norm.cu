// norm.cu -- residual addition, root-mean-square norm and per-token E4M3
// quantisation in one pass over the rows (what stands in front of the Q8
// linear of fp8.cu).
//
// Per row: h = bf16(x + r), y = h w rstd with rstd = 1 / sqrt(mean h^2 + eps),
// sa = max |y| / 448, xq = E4M3(y / sa).  With a = h w the quotient is
// a rstd / (max |a| rstd / 448) = a (448 / max |a|): the norm drops out of the
// codes, so ONE block reduction gives both the sum of squares and max |a|, and
// the row stays in registers between its single load and its stores.
// Bound: HBM (2 K read per input, 2 K written for h, K for the codes): 8192 x 4096
// with a residual in 36.0 us, 6.5 TB/s.  Two values per instruction and the products
// kept in registers for the codes (46.9 us with single ones formed twice: the
// issue slots were the bound).  288 rows of 3584: 3.3 us; one row of 4096: 1.7 us.
#include <algorithm>
#include <cmath>
#include <cuda_fp8.h>

#include "qspec_device.cuh"
#include "qspec_host.h"

namespace qspec {

namespace {

namespace nrm {

constexpr int kMaxK = 32768;

__device__ __forceinline__ float lo_f(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_f(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(b), "f"(a));
    return r;
}
__device__ __forceinline__ uint32_t add_bf16(uint32_t a, uint32_t b) {      // two bf16 sums, each rounded once
    uint32_t d;
    asm("add.rn.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
// two fp32 values in a register pair, and packed operations on them
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t both(uint32_t w) { return f2(lo_f(w), hi_f(w)); }
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
// two E4M3 codes, the first in the low byte
__device__ __forceinline__ uint32_t pack_e4m3(uint64_t v) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo32(v), hi32(v)), __NV_SATFINITE, __NV_E4M3);
}

// sum and maximum over the TPR threads of a row (all rows of a CTA take part)
template <int TPR>
__device__ __forceinline__ void row_reduce(float &sum, float &mx, float2 *red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) {
        sum += __shfl_xor_sync(0xffffffffu, sum, o);
        mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
    }
    if constexpr (TPR > 32) {
        constexpr int kW = TPR / 32;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        __syncthreads();                       // red free again (a second pass over the row)
        if (lane == 0) red[warp] = make_float2(sum, mx);
        __syncthreads();
        const float2 v = red[lane % kW];       // every warp folds the kW partials in the same order
        sum = v.x;
        mx = v.y;
#pragma unroll
        for (int o = kW / 2; o >= 1; o >>= 1) {
            sum += __shfl_xor_sync(0xffffffffu, sum, o);
            mx = max_nan(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        }
    }
}

// TPR threads per row, up to NV 16-byte words of a row per thread: as many threads
// as leave each two loads in flight per input, and a warp per row without a barrier
// where a row is short
template <int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR)
    rmsnorm_fp8_kernel(const uint16_t *x, int ldx, const uint16_t *res, int ldr,
                       const uint16_t *__restrict__ w, float eps, int M, int K, uint16_t *h, int ldh,
                       uint8_t *__restrict__ xq, float *__restrict__ sa, uint16_t *__restrict__ y, int ldy,
                       int32_t *st) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    __shared__ float2 red[32];
    const int t = threadIdx.x % TPR;
    const int m = blockIdx.x * kRows + (TPR < 128 ? threadIdx.x / TPR : 0);
    const int n8 = K / 8;
    const bool row_ok = m < M;
    pdl_launch_dependents();
    pdl_wait();
    uint4 hv[NV], wv[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = t + j * TPR;
        const bool in = row_ok && i < n8;
        hv[j] = in ? __ldcs(reinterpret_cast<const uint4 *>(x + (size_t)m * ldx) + i) : make_uint4(0, 0, 0, 0);
        wv[j] = in ? __ldg(reinterpret_cast<const uint4 *>(w) + i) : make_uint4(0, 0, 0, 0);
    }
    if (res != nullptr) {
        uint4 rv[NV];
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = t + j * TPR;
            rv[j] = row_ok && i < n8 ? __ldcs(reinterpret_cast<const uint4 *>(res + (size_t)m * ldr) + i)
                                     : make_uint4(0, 0, 0, 0);
        }
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            const int i = t + j * TPR;
            hv[j] = make_uint4(add_bf16(hv[j].x, rv[j].x), add_bf16(hv[j].y, rv[j].y), add_bf16(hv[j].z, rv[j].z),
                               add_bf16(hv[j].w, rv[j].w));
            if (row_ok && i < n8) reinterpret_cast<uint4 *>(h + (size_t)m * ldh)[i] = hv[j];
        }
    }
    // sum h^2 and max |h w|; the products stay in registers for the codes
    uint64_t a[NV][4], sq = 0;
    float amax = 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const uint32_t hw[4] = {hv[j].x, hv[j].y, hv[j].z, hv[j].w}, ww[4] = {wv[j].x, wv[j].y, wv[j].z, wv[j].w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t v = both(hw[e]);
            sq = fma2(v, v, sq);
            a[j][e] = mul2(v, both(ww[e]));
            amax = max_abs(amax, lo32(a[j][e]), hi32(a[j][e]));
        }
    }
    float ss = lo32(sq) + hi32(sq), down = 1.0f;
    row_reduce<TPR>(ss, amax, red);
    // Where the squares of finite values pass fp32 (|h| above 1e19), or the products
    // with large weights, the row is read and taken again times 2^-80.  A sum of
    // squares that did not pass it stands (times 2^-160 little would be left of it).
    const bool again = !(ss < INFINITY && amax < INFINITY), stands = ss < INFINITY;
    const float first = ss;
    if (TPR > 32 ? again : __any_sync(0xffffffffu, again)) {
        if (again) down = 8.271806125530277e-25f;        // 2^-80
        const uint16_t *row = res != nullptr ? h + (size_t)m * ldh : x + (size_t)m * ldx;
        ss = 0.0f;
        amax = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j) {
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * (t + j * TPR) + e;
                const bool in = row_ok && i < 4 * n8;
                const uint64_t v = mul2(both(in ? reinterpret_cast<const uint32_t *>(row)[i] : 0u), f2(down, down));
                ss = fmaf(lo32(v), lo32(v), fmaf(hi32(v), hi32(v), ss));
                a[j][e] = mul2(v, both(in ? reinterpret_cast<const uint32_t *>(w)[i] : 0u));
                amax = max_abs(amax, lo32(a[j][e]), hi32(a[j][e]));
            }
        }
        row_reduce<TPR>(ss, amax, red);
        if (stands) ss = first;
    }
    if (!row_ok) return;
    if (!(amax < INFINITY)) amax = INFINITY;             // (NaN too)
    const float of_ss = stands ? 1.0f : down;            // what ss was taken of: h times this
    const float rstd = rsqrtf(fmaf(ss, 1.0f / (float)K, eps * of_ss * of_ss)) * (of_ss == down ? 1.0f : 1.2089258196146292e24f);   // (2^80)
    // y = a rstd; codes a (448 / max |a|), where 448 / max |a| would pass fp32
    // with a brought up first
    const float up = amax < 1.0e-30f ? 7.9228162514264338e28f : 1.0f;   // 2^96
    const float inv = amax > 0.0f ? __fdiv_rn(448.0f, amax * up) : 0.0f;
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = t + j * TPR;
        if (i >= n8) continue;
        if (y != nullptr) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t v = mul2(a[j][e], f2(rstd, rstd));
                o[e] = pack_bf16(lo32(v), hi32(v));
            }
            reinterpret_cast<uint4 *>(y + (size_t)m * ldy)[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
        uint32_t code[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (up != 1.0f) a[j][e] = mul2(a[j][e], f2(up, up));
            code[e] = pack_e4m3(mul2(a[j][e], f2(inv, inv)));
        }
        reinterpret_cast<uint2 *>(xq + (size_t)m * K)[i] =
            amax > 0.0f ? make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16)
                        : make_uint2(0u, 0u);         // no code of -0 in a row of zeros
    }
    if (t == 0) {
        const float top = amax * rstd, s = __fdiv_rn(top, 448.0f);          // max |y|, in the bf16 output inf from the
        sa[m] = s;                                                           // midpoint behind the largest bf16 value
        if (!(ss < INFINITY) || !(top < (y != nullptr ? 3.3961775292304601e38f : INFINITY))) flag(st, QSPEC_ERR_NONFINITE);
    }
}

template <int TPR, int NV>
int launch(const uint16_t *x, int ldx, const uint16_t *res, int ldr, const uint16_t *w, float eps, int M, int K,
           uint16_t *h, int ldh, uint8_t *xq, float *sa, uint16_t *y, int ldy, int32_t *st, cudaStream_t stream) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    return launch_pdl("qspec_rmsnorm_fp8", rmsnorm_fp8_kernel<TPR, NV>, dim3((unsigned)((M + kRows - 1) / kRows)),
                      dim3(TPR < 128 ? 128 : TPR), 0, stream, x, ldx, res, ldr, w, eps, M, K, h, ldh, xq, sa, y, ldy,
                      st);
}

}  // namespace nrm

}  // namespace

}  // namespace qspec

using namespace qspec;

extern "C" int qspec_rmsnorm_fp8(const uint16_t *x_bf16, int ldx, const uint16_t *res_bf16, int ldr,
                                 const uint16_t *w_bf16, float eps, int M, int K, uint16_t *h_bf16, int ldh,
                                 uint8_t *xq, float *sa, uint16_t *y_bf16, int ldy, int32_t *dev_status,
                                 qspec_stream_t stream) {
    if (!x_bf16 || !w_bf16 || !xq || !sa || (res_bf16 != nullptr) != (h_bf16 != nullptr)) return QSPEC_ERR_NULL;
    if (M < 1 || K < kGroup || K % kGroup || K > nrm::kMaxK || !(eps > 0.0f) || !std::isfinite(eps) || ldx < K ||
        (res_bf16 && (ldr < K || ldh < K)) || (y_bf16 && ldy < K))
        return QSPEC_ERR_SHAPE;
    if (!aligned(x_bf16, 16) || !aligned(w_bf16, 16) || !aligned(xq, 8) || !aligned(sa, 4) || ldx % 8 ||
        (res_bf16 && (!aligned(res_bf16, 16) || !aligned(h_bf16, 16) || ldr % 8 || ldh % 8)) ||
        (y_bf16 && (!aligned(y_bf16, 16) || ldy % 8)))
        return QSPEC_ERR_ALIGN;
    int rc = check_device();
    if (rc) return rc;
    cudaStream_t s = as_cuda(stream);
    auto go = [&](auto launcher) {
        return launcher(x_bf16, ldx, res_bf16, ldr, w_bf16, eps, M, K, h_bf16, ldh, xq, sa, y_bf16, ldy, dev_status,
                        s);
    };
    const int n8 = K / 8;
    if (n8 <= 128) return go(nrm::launch<32, 4>);
    if (n8 <= 512) return go(nrm::launch<256, 2>);
    if (n8 <= 1024) return go(nrm::launch<512, 2>);
    if (n8 <= 2048) return go(nrm::launch<1024, 2>);
    return go(nrm::launch<1024, 4>);
}
