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

#include "fp8_block.cuh"
#include "qspec_host.h"

namespace qspec {

namespace {

namespace nrm {

using f8b::f2;
using f8b::fma2;
using f8b::hi32;
using f8b::lo32;
using f8b::max_abs;
using f8b::max_nan;
using f8b::mul2;

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
__device__ __forceinline__ uint64_t both(uint32_t w) { return f2(lo_f(w), hi_f(w)); }
// two E4M3 codes, the first in the low byte
__device__ __forceinline__ uint32_t pack_e4m3(uint64_t v) {
    return __nv_cvt_float2_to_fp8x2(make_float2(lo32(v), hi32(v)), __NV_SATFINITE, __NV_E4M3);
}

// Eight codes of y = h w rstd over a scale s as it is stored, where that is a subnormal number or 0 (there the codes by
// 448 / max |a| belong to the scale before its last rounding); a product h w may be below fp32 too.  In place of the
// codes stored before, by the thread that did so: looking for such blocks in front of them took 3 to 11 % of the call.
__device__ __forceinline__ void recode(const uint4 *h, const uint4 *w, float rstd, float s, uint2 *xq) {
    const uint4 hv = *h, wv = *w;
    const uint32_t hw[4] = {hv.x, hv.y, hv.z, hv.w}, ww[4] = {wv.x, wv.y, wv.z, wv.w};
    const double by = (double)rstd * (double)__frcp_rn(s * 0x1p100f) * 0x1p100;
    uint32_t code[4];
#pragma unroll
    for (int e = 0; e < 4; ++e)
        code[e] = s > 0.0f ? pack_e4m3(f2((float)((double)lo_f(hw[e]) * (double)lo_f(ww[e]) * by), (float)((double)hi_f(hw[e]) * (double)hi_f(ww[e]) * by))) : 0u;
    *xq = make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
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
    const float top = amax * rstd;                       // max |y|, in the bf16 output inf from the midpoint behind the largest bf16 value
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
            top <= f8b::kNothing ? make_uint2(0u, 0u)            // beside a scale of 0, of a row of zeros among them: no code, nor -0
                                 : make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16);
    }
    if (t == 0) {
        sa[m] = __fdiv_rn(top, 448.0f);
        if (!(ss < INFINITY) || !(top < (y != nullptr ? 3.3961775292304601e38f : INFINITY))) flag(st, QSPEC_ERR_NONFINITE);
    }
}

// The same with a scale for each block of 128: half a warp holds a block (16 lanes x 8 values), so its maximum takes
// four shuffles and the row's reduction only the sum of squares.  Where the squares pass fp32 the sum is taken again
// times 2^-160; a block whose products with the weights pass it is taken again times 2^-80, the other blocks stand.
// Scales lie token by token, [K / 128][lds]: 4 bytes a block, next to those of the neighbouring rows' CTAs.
//
// Many rows take half the threads and twice the words to each (NV = 4, 1024 threads to an SM): more rows at once, each with
// twice the loads in flight.  A thread's odd words are summed apart, as the thread does that has them in the wide form, so
// that a row's bits do not depend on the number of rows.
template <int TPR, int NV>
constexpr bool kNarrow = NV == 4 && TPR >= 128 && TPR < 1024;
template <int TPR, int NV>                     // CTAs to an SM
constexpr int kOcc = kNarrow<TPR, NV> ? 1024 / TPR : NV == 2 && TPR == 256 ? 5 : NV == 2 && TPR == 512 ? 3 : 1;

template <int TPR, int S>
__device__ __forceinline__ float row_sum(float (&part)[S], float *red) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1)
#pragma unroll
        for (int i = 0; i < S; ++i) part[i] += __shfl_xor_sync(0xffffffffu, part[i], o);
    float sum = S == 2 ? part[0] + part[S - 1] : part[0];
    if constexpr (TPR > 32) {
        constexpr int kW = TPR / 32;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
        __syncthreads();                       // red free again (a second pass over the row)
        if (lane == 0) red[warp] = sum;
        __syncthreads();
        sum = red[lane % kW];                  // every warp folds the kW partials in the same order
#pragma unroll
        for (int o = kW / 2; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    }
    return sum;
}

template <int TPR, int NV>
__global__ void __launch_bounds__(TPR < 128 ? 128 : TPR, (kOcc<TPR, NV>))
    rmsnorm_fp8_block_kernel(const uint16_t *x, int ldx, const uint16_t *res, int ldr, const uint16_t *__restrict__ w,
                             float eps, int M, int K, uint16_t *h, int ldh, uint8_t *__restrict__ xq,
                             float *__restrict__ sa, int lds, uint16_t *__restrict__ y, int ldy, int32_t *st) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    constexpr float kDown = 8.271806125530277e-25f, kUp = 1.2089258196146292e24f;      // 2^-80, 2^80
    constexpr int S = kNarrow<TPR, NV> ? 2 : 1;
    __shared__ float red[32];
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
    uint64_t a[NV][4], sq[S] = {};
    float top[NV];
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const uint32_t hw[4] = {hv[j].x, hv[j].y, hv[j].z, hv[j].w}, ww[4] = {wv[j].x, wv[j].y, wv[j].z, wv[j].w};
        top[j] = 0.0f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint64_t v = both(hw[e]);
            sq[j % S] = fma2(v, v, sq[j % S]);
            a[j][e] = mul2(v, both(ww[e]));
            top[j] = max_abs(top[j], lo32(a[j][e]), hi32(a[j][e]));
        }
#pragma unroll
        for (int o = 8; o >= 1; o >>= 1) top[j] = max_nan(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
    }
    float part[S];
#pragma unroll
    for (int i = 0; i < S; ++i) part[i] = lo32(sq[i]) + hi32(sq[i]);
    float ss = row_sum<TPR>(part, red);
    const uint16_t *row = res != nullptr ? h + (size_t)m * ldh : x + (size_t)m * ldx;
    const bool stands = ss < INFINITY;                    // (the same for a row's threads, and for TPR = 32 for a warp's)
    if (!stands) {
#pragma unroll
        for (int i = 0; i < S; ++i) part[i] = 0.0f;
#pragma unroll
        for (int j = 0; j < NV; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const int i = 4 * (t + j * TPR) + e;
                const uint64_t v = mul2(both(row_ok && i < 4 * n8 ? reinterpret_cast<const uint32_t *>(row)[i] : 0u), f2(kDown, kDown));
                part[j % S] = fmaf(lo32(v), lo32(v), fmaf(hi32(v), hi32(v), part[j % S]));
            }
        ss = row_sum<TPR>(part, red);
    }
    if (!row_ok) return;                                  // (whole warps: a row has at least one)
    const float near = rsqrtf(fmaf(ss, 1.0f / (float)K, stands ? eps : eps * kDown * kDown));
    // 1 / rms, for products as they are and for those times 2^-80
    const float rstd = stands ? near : near * kDown, rstd_up = stands ? near * kUp : near;
    bool bad = !(ss < INFINITY), any = false;
    uint32_t again = 0, low = 0;                          // bit j: block j was taken again; has a subnormal scale, or one of 0
#pragma unroll
    for (int j = 0; j < NV; ++j) any |= !(top[j] < INFINITY);
    if (__any_sync(0xffffffffu, any)) {
#pragma unroll
        for (int j = 0; j < NV; ++j) {
            if (!(top[j] < INFINITY)) {
                again |= 1u << j;
                top[j] = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int at = 4 * (t + j * TPR) + e;
                    const bool in = at < 4 * n8;
                    a[j][e] = mul2(mul2(both(in ? reinterpret_cast<const uint32_t *>(row)[at] : 0u), f2(kDown, kDown)),
                                   both(in ? reinterpret_cast<const uint32_t *>(w)[at] : 0u));
                    top[j] = max_abs(top[j], lo32(a[j][e]), hi32(a[j][e]));
                }
            }
#pragma unroll
            for (int o = 8; o >= 1; o >>= 1) top[j] = max_nan(top[j], __shfl_xor_sync(0xffffffffu, top[j], o));
            if (!(top[j] < INFINITY)) top[j] = INFINITY;          // (NaN too)
        }
    }
#pragma unroll
    for (int j = 0; j < NV; ++j) {
        const int i = t + j * TPR;
        const float by = again >> j & 1 ? rstd_up : rstd;
        if (i >= n8) continue;
        if (y != nullptr) {
            uint32_t o[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint64_t v = mul2(a[j][e], f2(by, by));
                o[e] = pack_bf16(lo32(v), hi32(v));
            }
            reinterpret_cast<uint4 *>(y + (size_t)m * ldy)[i] = make_uint4(o[0], o[1], o[2], o[3]);
        }
        // codes a (448 / top), within 3 x 2^-24; a power of two beside them where the reciprocal would leave fp32
        const float up = f8b::lift(top[j]);
        const float inv = 448.0f * f8b::reciprocal(top[j] * up);
        uint32_t code[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            if (up != 1.0f) a[j][e] = mul2(a[j][e], f2(up, up));
            code[e] = pack_e4m3(mul2(a[j][e], f2(inv, inv)));
        }
        reinterpret_cast<uint2 *>(xq + (size_t)m * K)[i] =
            top[j] > 0.0f ? make_uint2(code[0] | code[1] << 16, code[2] | code[3] << 16)
                          : make_uint2(0u, 0u);       // no code, nor -0, in a block of zeros
        const float most = top[j] * by;                // max |y|, in the bf16 output inf from the midpoint behind the
        bad |= !(most < (y != nullptr ? 3.3961775292304601e38f : INFINITY));   // largest bf16 value
        low |= top[j] > 0.0f && most < f8b::kSubnormal ? 1u << j : 0u;
        if ((threadIdx.x & 15) == 0) sa[(size_t)(i / 16) * lds + m] = f8b::scale_of(most);
    }
    if (low != 0) {
#pragma unroll
        for (int j = 0; j < NV; ++j)
            if (low >> j & 1) {
                const int i = t + j * TPR;
                recode(reinterpret_cast<const uint4 *>(row) + i, reinterpret_cast<const uint4 *>(w) + i, rstd, f8b::scale_of(top[j] * rstd),
                       reinterpret_cast<uint2 *>(xq + (size_t)m * K) + i);
            }
    }
    if (__any_sync(0xffffffffu, bad) && (threadIdx.x & 31) == 0) flag(st, QSPEC_ERR_NONFINITE);
}

template <int TPR, int NV>
int launch(const uint16_t *x, int ldx, const uint16_t *res, int ldr, const uint16_t *w, float eps, int M, int K,
           uint16_t *h, int ldh, uint8_t *xq, float *sa, uint16_t *y, int ldy, int32_t *st, cudaStream_t stream) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    return launch_pdl("qspec_rmsnorm_fp8", rmsnorm_fp8_kernel<TPR, NV>, dim3((unsigned)((M + kRows - 1) / kRows)),
                      dim3(TPR < 128 ? 128 : TPR), 0, stream, x, ldx, res, ldr, w, eps, M, K, h, ldh, xq, sa, y, ldy,
                      st);
}

template <int TPR, int NV>
int launch_block(const uint16_t *x, int ldx, const uint16_t *res, int ldr, const uint16_t *w, float eps, int M, int K,
                 uint16_t *h, int ldh, uint8_t *xq, float *sa, int lds, uint16_t *y, int ldy, int32_t *st,
                 cudaStream_t stream) {
    constexpr int kRows = TPR < 128 ? 128 / TPR : 1;
    return launch_pdl("qspec_rmsnorm_fp8_block", rmsnorm_fp8_block_kernel<TPR, NV>,
                      dim3((unsigned)((M + kRows - 1) / kRows)), dim3(TPR < 128 ? 128 : TPR), 0, stream, x, ldx, res,
                      ldr, w, eps, M, K, h, ldh, xq, sa, lds, y, ldy, st);
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

extern "C" int qspec_rmsnorm_fp8_block(const uint16_t *x_bf16, int ldx, const uint16_t *res_bf16, int ldr,
                                 const uint16_t *w_bf16, float eps, int M, int K, uint16_t *h_bf16, int ldh,
                                 uint8_t *xq, float *sa, int lds, uint16_t *y_bf16, int ldy, int32_t *dev_status,
                                 qspec_stream_t stream) {
    if (!x_bf16 || !w_bf16 || !xq || !sa || (res_bf16 != nullptr) != (h_bf16 != nullptr)) return QSPEC_ERR_NULL;
    if (M < 1 || K < kGroup || K % kGroup || K > nrm::kMaxK || !(eps > 0.0f) || !std::isfinite(eps) || ldx < K ||
        lds < M ||
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
        return launcher(x_bf16, ldx, res_bf16, ldr, w_bf16, eps, M, K, h_bf16, ldh, xq, sa, lds, y_bf16, ldy, dev_status,
                        s);
    };
    // Widths as in qspec_rmsnorm_fp8, halved where the rows fill the device even so.  (us, wide / halved, with residual and y:
    // 2047 x 3584 10.6 / 10.1, 8192 x 2048 29.5 / 25.2, 2047 x 5120 17.4 / 15.1, 8192 x 14336 201 / 157, but 912 x 4096 6.7 /
    // 6.9, 456 x 8192 6.7 / 7.1, 64 x 14336 3.5 / 4.0; since then a twentieth less by scales without divisions.)
    const int n8 = K / 8;
    const auto many = [&](int threads) { return (long long)M * threads >= 1024LL * sm_count(); };
    if (n8 <= 128) return go(nrm::launch_block<32, 4>);
    if (n8 <= 512 && many(128)) return go(nrm::launch_block<128, 4>);
    if (n8 > 512 && n8 <= 1024 && many(256)) return go(nrm::launch_block<256, 4>);
    if (n8 > 1024 && n8 <= 2048 && many(512)) return go(nrm::launch_block<512, 4>);
    if (n8 <= 512) return go(nrm::launch_block<256, 2>);
    if (n8 <= 1024) return go(nrm::launch_block<512, 2>);
    if (n8 <= 2048) return go(nrm::launch_block<1024, 2>);
    return go(nrm::launch_block<1024, 4>);
}
