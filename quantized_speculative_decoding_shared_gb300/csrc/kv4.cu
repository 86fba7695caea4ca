// kv4.cu -- rows into and out of the 4-bit KV cache.
//
// Per (row, head): lo = min(0, min x), hi = max(0, max x), s = fp16((hi - lo) / 15),
// z = clamp(rint(-lo / s), 0, 15), code = clamp(rint(x / s) + z, 0, 15); 0 is in the
// range, so it keeps an exact code.  The quotient x / s is one Newton step
// from q0 = x y, y = 1 / s: fma(fma(-q0, s, x), y, q0).  x has 8 significant bits
// and s 11, so x / s is either a half-integer exactly (then the step returns
// it exactly) or at least 2^-10 from one for |x / s| < 16 (far beyond the
// step's error): rint gives what the IEEE quotient gives.
//
// Pure streaming, bound by HBM: 16 bytes (8 values) per thread, D / 8 threads
// per head row, K and V in the same thread so that a row's two loads overlap.
#include <algorithm>
#include <cuda_fp16.h>

#include "qspec_device.cuh"
#include "qspec_host.h"

namespace qspec {

namespace {

namespace kv4 {

constexpr int kThreads = 256;

struct Rows {
    const int32_t *start, *base;
    int rows, B, H, T;
};

// The position of packed row m in its sequence b, or -1: rows of no sequence,
// and sequences whose ranges do not hold (flagged at the sequence's first row).
__device__ __forceinline__ int locate(const Rows &r, int m, int &b) {
    int lo = 0, hi = r.B;                        // last b with start[b] <= m
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(r.start + mid) <= m)
            lo = mid;
        else
            hi = mid;
    }
    b = lo;
    const int s0 = __ldg(r.start + lo), s1 = __ldg(r.start + lo + 1), p0 = __ldg(r.base + lo);
    if (m < s0 || m >= s1 || s0 < 0 || s1 > r.rows || p0 < 0 || (long long)p0 + (s1 - s0) > r.T) return -1;
    return p0 + (m - s0);
}

// every sequence's ranges, by the first CTA (so that one without rows of its
// own in the launch is reported too)
__device__ __forceinline__ void check_ranges(const Rows &r, int32_t *st) {
    if (blockIdx.x != 0) return;
    bool bad = false;
    for (int b = threadIdx.x; b < r.B; b += kThreads) {
        const int s0 = r.start[b], s1 = r.start[b + 1], p0 = r.base[b];
        bad |= s0 < 0 || s1 < s0 || s1 > r.rows || p0 < 0 || (long long)p0 + ((long long)s1 - s0) > r.T;
    }
    if (bad) flag(st, QSPEC_ERR_RANGE);
}

// 8 values of a head row held by L = D / 8 consecutive lanes -> their codes as
// nibbles, and the row's scale word
template <int L>
__device__ __forceinline__ uint32_t quantise(const uint4 &v, uint32_t &word, bool &bad) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    float f[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        f[2 * i] = __uint_as_float(w[i] << 16);
        f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    float lo = 0.0f, hi = 0.0f;
    bool nan = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        lo = fminf(lo, f[i]);
        hi = fmaxf(hi, f[i]);
        nan |= f[i] != f[i];
    }
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) {
        lo = fminf(lo, __shfl_xor_sync(0xffffffffu, lo, o));
        hi = fmaxf(hi, __shfl_xor_sync(0xffffffffu, hi, o));
    }
    const __half sh = __float2half_rn(__fdiv_rn(__fsub_rn(hi, lo), 15.0f));
    const float s = __half2float(sh);
    bad |= nan || !(s < INFINITY);
    const float y = s > 0.0f ? __frcp_rn(s) : 0.0f;
    auto quot = [&](float x) {
        const float q0 = __fmul_rn(x, y);
        return rintf(__fmaf_rn(__fmaf_rn(-q0, s, x), y, q0));
    };
    const float z = s > 0.0f ? fminf(fmaxf(quot(-lo), 0.0f), 15.0f) : 0.0f;
    uint32_t nib = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float c = s > 0.0f ? fminf(fmaxf(quot(f[i]) + z, 0.0f), 15.0f) : 0.0f;
        nib |= (uint32_t)(int)c << (4 * i);
    }
    word = (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(__float2half_rn(z)) << 16);
    return nib;
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    append_kernel(const uint16_t *__restrict__ k, int ldk, const uint16_t *__restrict__ v, int ldv, Rows r,
                  uint32_t *__restrict__ kc, uint32_t *__restrict__ ks, uint32_t *__restrict__ vc,
                  uint32_t *__restrict__ vs, int32_t *st) {
    constexpr int L = D / 8;
    pdl_launch_dependents();
    pdl_wait();
    check_ranges(r, st);
    const long long item = ((long long)blockIdx.x * kThreads + threadIdx.x) / L;
    const int l = threadIdx.x % L;
    const int m = (int)(item / r.H), hd = (int)(item - (long long)m * r.H);
    int b = 0;
    const int pos = m < r.rows ? locate(r, m, b) : -1;
    uint4 kv = make_uint4(0, 0, 0, 0), vv = kv;
    if (pos >= 0) {
        kv = __ldcs(reinterpret_cast<const uint4 *>(k + (size_t)m * ldk + (size_t)hd * D) + l);
        vv = __ldcs(reinterpret_cast<const uint4 *>(v + (size_t)m * ldv + (size_t)hd * D) + l);
    }
    bool bad = false;
    uint32_t kw, vw;
    const uint32_t kn = quantise<L>(kv, kw, bad), vn = quantise<L>(vv, vw, bad);
    if (pos >= 0) {
        const size_t at = ((size_t)b * r.H + hd) * r.T + pos;
        kc[at * L + l] = kn;
        vc[at * L + l] = vn;
        if (l == 0) {
            ks[at] = kw;
            vs[at] = vw;
        }
    }
    if (bad) flag(st, QSPEC_ERR_NONFINITE);
}

// 8 codes and a scale word -> 8 bf16 values s (c - z), each rounded once (the
// product of an fp16 and a 4-bit integer is exact in fp32)
__device__ __forceinline__ uint4 values(uint32_t nib, uint32_t word) {
    const float s = __half2float(__ushort_as_half((uint16_t)(word & 0xFFFFu)));
    const float z = __half2float(__ushort_as_half((uint16_t)(word >> 16)));
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = s * ((float)((nib >> (8 * i)) & 15u) - z), c = s * ((float)((nib >> (8 * i + 4)) & 15u) - z);
        o[i] = (uint32_t)float_to_bf16_bits(a) | ((uint32_t)float_to_bf16_bits(c) << 16);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    load_kernel(const uint32_t *__restrict__ kc, const uint32_t *__restrict__ ks, const uint32_t *__restrict__ vc,
                const uint32_t *__restrict__ vs, Rows r, uint16_t *__restrict__ k, int ldk, uint16_t *__restrict__ v,
                int ldv, int32_t *st) {
    constexpr int L = D / 8;
    pdl_launch_dependents();
    pdl_wait();
    check_ranges(r, st);
    const long long item = ((long long)blockIdx.x * kThreads + threadIdx.x) / L;
    const int l = threadIdx.x % L;
    const int m = (int)(item / r.H), hd = (int)(item - (long long)m * r.H);
    if (m >= r.rows) return;
    int b = 0;
    const int pos = locate(r, m, b);
    if (pos < 0) return;
    const size_t at = ((size_t)b * r.H + hd) * r.T + pos;
    const uint32_t kn = kc[at * L + l], vn = vc[at * L + l], kw = ks[at], vw = vs[at];
    reinterpret_cast<uint4 *>(k + (size_t)m * ldk + (size_t)hd * D)[l] = values(kn, kw);
    reinterpret_cast<uint4 *>(v + (size_t)m * ldv + (size_t)hd * D)[l] = values(vn, vw);
}

// what both calls can refuse on the host
int check(const void *k, int ldk, const void *v, int ldv, const int32_t *start, const int32_t *base, int rows, int B,
          int H, int T, int D, const void *kc, const void *ks, const void *vc, const void *vs) {
    if (!start || !base || !kc || !ks || !vc || !vs || (rows > 0 && (!k || !v))) return QSPEC_ERR_NULL;
    if (rows < 0 || B < 1 || H < 1 || T < 1 || (D != 64 && D != 128)) return QSPEC_ERR_SHAPE;
    if (ldk < (long long)H * D || ldv < (long long)H * D) return QSPEC_ERR_SHAPE;
    if ((long long)rows * H * (D / 8) / kThreads >= (1LL << 31) - 1) return QSPEC_ERR_SHAPE;
    if (ldk % 8 || ldv % 8 || !aligned(k, 16) || !aligned(v, 16) || !aligned(kc, 16) || !aligned(vc, 16) ||
        !aligned(ks, 4) || !aligned(vs, 4) || !aligned(start, 4) || !aligned(base, 4))
        return QSPEC_ERR_ALIGN;
    return check_device();
}

}  // namespace kv4

}  // namespace

}  // namespace qspec

using namespace qspec;

extern "C" int qspec_kv4_append(const uint16_t *k_bf16, int ldk, const uint16_t *v_bf16, int ldv,
                                const int32_t *row_start, const int32_t *base_pos, int rows, int B, int H, int T,
                                int D, uint8_t *k_codes, uint32_t *k_sz, uint8_t *v_codes, uint32_t *v_sz,
                                int32_t *dev_status, qspec_stream_t stream) {
    int rc = kv4::check(k_bf16, ldk, v_bf16, ldv, row_start, base_pos, rows, B, H, T, D, k_codes, k_sz, v_codes, v_sz);
    if (rc || rows == 0) return rc;
    const kv4::Rows r{row_start, base_pos, rows, B, H, T};
    const unsigned grid = (unsigned)(((long long)rows * H * (D / 8) + kv4::kThreads - 1) / kv4::kThreads);
    auto kern = D == 128 ? kv4::append_kernel<128> : kv4::append_kernel<64>;
    return launch_pdl("qspec_kv4_append", kern, dim3(grid), dim3(kv4::kThreads), 0, as_cuda(stream), k_bf16, ldk,
                      v_bf16, ldv, r, reinterpret_cast<uint32_t *>(k_codes), k_sz,
                      reinterpret_cast<uint32_t *>(v_codes), v_sz, dev_status);
}

extern "C" int qspec_kv4_load(const uint8_t *k_codes, const uint32_t *k_sz, const uint8_t *v_codes,
                              const uint32_t *v_sz, const int32_t *row_start, const int32_t *base_pos, int rows,
                              int B, int H, int T, int D, uint16_t *k_bf16, int ldk, uint16_t *v_bf16, int ldv,
                              int32_t *dev_status, qspec_stream_t stream) {
    int rc = kv4::check(k_bf16, ldk, v_bf16, ldv, row_start, base_pos, rows, B, H, T, D, k_codes, k_sz, v_codes, v_sz);
    if (rc || rows == 0) return rc;
    const kv4::Rows r{row_start, base_pos, rows, B, H, T};
    const unsigned grid = (unsigned)(((long long)rows * H * (D / 8) + kv4::kThreads - 1) / kv4::kThreads);
    auto kern = D == 128 ? kv4::load_kernel<128> : kv4::load_kernel<64>;
    return launch_pdl("qspec_kv4_load", kern, dim3(grid), dim3(kv4::kThreads), 0, as_cuda(stream),
                      reinterpret_cast<const uint32_t *>(k_codes), k_sz, reinterpret_cast<const uint32_t *>(v_codes),
                      v_sz, r, k_bf16, ldk, v_bf16, ldv, dev_status);
}
