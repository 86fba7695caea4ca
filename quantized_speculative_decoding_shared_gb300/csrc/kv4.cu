// kv4.cu -- rows into and out of the 4-bit KV cache.
//
// Per (row, head): lo = min(0, min x), hi = max(0, max x), s = fp16((hi - lo) / 15),
// z = clamp(rint(-lo / s), 0, 15), code = clamp(rint(x / s) + z, 0, 15); 0 is in the
// range, so it keeps an exact code.  The quotient x / s is one Newton step
// from q0 = x y, y = 1 / s: fma(fma(-q0, s, x), y, q0).  x = X 2^a has 8 significant
// bits and s = S 2^b 11, so x / s is either a half-integer exactly (then the step
// returns it exactly) or at least 1 / 4094 from one, that is |2 X 2^a - (2 n + 1) S 2^b| / (2 S 2^b)
// at its least (S = 2047, a = b + 3; over all X, S and a - b).  The step is off by some
// 2^-19 where |x / s| < 32: rint gives what the IEEE quotient gives.  Quotients of 16 and more
// come with scales that are fp16 subnormals only, and end at the clamp.
//
// Streaming: 2 D bytes of a head row against D / 2 + 4 of the cache.  Long prompts
// come to HBM's rate on the way out (32764 rows of 8 heads of 128: load 6.2 TB/s,
// append 4.6).  At 8191 rows (11.7 us in, 8.9 out) neither the issue slots (65 % used in
// append) nor DRAM (28 %) is the bound but the way through a short-lived warp: a
// search and its loads' latency in front of four head rows.  A warp takes one head
// of R consecutive rows of K and of V, L = D / 8 lanes to a head row, 16 bytes (8
// values) to a lane and kRounds rows one after another: its codes and its scale
// words are then runs of positions in the cache, the rows are looked up once, and
// the loads of all rounds are in flight together.
#include <algorithm>
#include <climits>
#include <cuda_fp16.h>

#include "qspec_device.cuh"
#include "qspec_host.h"

namespace qspec {

namespace {

namespace kv4 {

constexpr int kThreads = 128, kWarps = kThreads / 32;
// head rows per group of lanes, of K and of V each: 8191 rows of 8 heads append in 11.7 us and load in 8.9 (four rounds:
// 11.3 and 9.9), 80 rows in 2.3 and 2.3 (2.9 and 2.5); 8 warps a CTA the same within 0.2, 2 warps 1.5 us slower
constexpr int kRounds = 2;
constexpr int kStage = 1024;                     // sequences whose starts are searched in shared memory

struct Rows {
    const int32_t *start, *base;
    int rows, B, H, T;
};

// what a warp works on, and its lanes' share of it
template <int D>
struct Part {
    static constexpr int L = D / 8, G = 32 / L, R = G * kRounds;
    int m0, hd, l, g;
    bool in;                                     // there are such rows

    __device__ __forceinline__ Part(const Rows &r) {
        const uint32_t unit = blockIdx.x * kWarps + (threadIdx.x >> 5), block = unit / (uint32_t)r.H;
        const int lane = threadIdx.x & 31;
        hd = (int)(unit - block * (uint32_t)r.H);
        in = (long long)block * R < r.rows;
        m0 = in ? (int)block * R : 0;
        l = lane % L;
        g = lane / L;
    }
    // the packed row of round i (of lanes j = 0 .. R - 1 that look the rows up: place j)
    __device__ __forceinline__ int row(int i) const { return m0 + g * kRounds + i; }
};

// the sequences' first rows into shared memory; a binary search there is short
// against one in global memory, whose steps each wait for the last
__device__ __forceinline__ const int32_t *stage_starts(const Rows &r, int32_t *buf) {
    if (r.B > kStage) return r.start;
    for (int i = threadIdx.x; i <= r.B; i += kThreads) buf[i] = __ldg(r.start + i);
    __syncthreads();
    return buf;
}

// The place (sequence, head, position) of packed row m in the cache if sequence b has it, or -1 (sequences
// whose ranges do not hold, flagged by check_ranges, have none).
__device__ __forceinline__ long long place_in(const Rows &r, const int32_t *start, int b, int m, int hd) {
    const int s0 = start[b], s1 = start[b + 1], p0 = __ldg(r.base + b);
    if (m < s0 || m >= s1 || s0 < 0 || s1 > r.rows || p0 < 0 || (long long)p0 + (s1 - s0) > r.T) return -1;
    return ((long long)b * r.H + hd) * r.T + p0 + (m - s0);
}
// The places of a warp's rows that a search has not found (lanes `lost`).  A start that does not hold can lead it
// past a row's sequence: the lanes look at all of them then.  Where the starts increase there is nothing to look
// for (rows of no sequence are what a caller may fill up with: 8192 of them append in 11.0 us at 16 sequences and
// 16.1 at 1000, 14.1 and 85 when looked for).
template <int R>
__device__ __forceinline__ long long look_through(const Rows &r, const int32_t *start, int m0, int hd, long long found, uint32_t lost) {
    const int lane = threadIdx.x & 31;
    bool increase = true;
#pragma unroll 4
    for (int b = lane; b < r.B; b += 32) increase &= start[b] <= start[b + 1];
    if (__all_sync(0xffffffffu, increase)) return found;
    for (int b0 = 0; b0 < r.B && lost; b0 += 32)
#pragma unroll 1
        for (int j = 0; j < R; ++j) {
            if (!(lost >> j & 1)) continue;
            long long at = b0 + lane < r.B ? place_in(r, start, b0 + lane, m0 + j, hd) : -1;
            const uint32_t has = __ballot_sync(0xffffffffu, at >= 0);
            if (has == 0) continue;
            at = __shfl_sync(0xffffffffu, at, __ffs(has) - 1);
            if (lane == j) found = at;
            lost &= ~(1u << j);
        }
    return found;
}
// Of lane j < R the place of row m0 + j, or -1: rows of no sequence.
template <int R>
__device__ __forceinline__ long long locate(const Rows &r, const int32_t *start, int m0, int hd) {
    const int lane = threadIdx.x & 31, m = m0 + lane;
    const bool mine = lane < R && m < r.rows;
    int lo = 0, hi = mine ? r.B : 0;             // last b with start[b] <= m
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (start[mid] <= m)
            lo = mid;
        else
            hi = mid;
    }
    const long long found = mine ? place_in(r, start, lo, m, hd) : -1;
    const uint32_t lost = __ballot_sync(0xffffffffu, mine && found < 0);
    return lost ? look_through<R>(r, start, m0, hd, found, lost) : found;
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

__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {          // of two bf16 values each, keeps a NaN
    uint32_t d;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(d) : "r"(a), "r"(b));
    return d;
}
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
    uint64_t d;
    asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(a), "l"(b), "l"(c));
    return d;
}
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
__device__ __forceinline__ float lo32(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi32(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }

// 8 values of a head row held by L consecutive lanes -> their codes as nibbles,
// and the row's scale word
template <int L>
__device__ __forceinline__ uint32_t quantise(const uint4 &v, uint32_t &word, bool &bad) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    // (max(0, -min), max(0, max)) as two bf16 values, exact
    const uint32_t n = 0x80008000u;
    const uint32_t top = max2(max2(w[0], w[1]), max2(w[2], w[3]));
    const uint32_t low = max2(max2(w[0] ^ n, w[1] ^ n), max2(w[2] ^ n, w[3] ^ n));
    uint32_t ends = max2(max2(__byte_perm(low, top, 0x5410), __byte_perm(low, top, 0x7632)), 0u);
#pragma unroll
    for (int o = L / 2; o >= 1; o >>= 1) ends = max2(ends, __shfl_xor_sync(0xffffffffu, ends, o));
    const float below = __uint_as_float(ends << 16), above = __uint_as_float(ends & 0xFFFF0000u);
    // (hi - lo) / 15, correctly rounded where it is a normal number (and 0 in fp16 where it is not): the residual
    // of the product with the rounded 1 / 15 is exact, and one step with it rounds like the quotient
    const float range = __fadd_rn(above, below), t0 = __fmul_rn(range, 1.0f / 15.0f);
    const __half sh = __float2half_rn(__fmaf_rn(__fmaf_rn(t0, -15.0f, range), 1.0f / 15.0f, t0));
    const float s = __half2float(sh);            // NaN where a value is not finite
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(s));
    if (!(s > 0.0f)) y = 0.0f;
    // rint by the addition of 1.5 x 2^23: the integer is then in the low bits.  q stays below 32: s is at
    // least half of (hi - lo) / 15 where it is not 0
    constexpr float kInt = 12582912.0f;
    auto quot = [&](uint64_t x) {
        const uint64_t q0 = mul2(x, f2(y, y));
        return add2(fma2(fma2(q0, f2(-s, -s), x), f2(y, y), q0), f2(kInt, kInt));
    };
    const uint32_t z = s > 0.0f ? (uint32_t)min((int)(__float_as_uint(lo32(quot(f2(below, below)))) & 0xFFu), 15) : 0u;
    // integers i and i + 4 of the eight in one register, then shifted in by nibbles
    uint32_t c[4];
    uint64_t t[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = quot(f2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u)));
    const uint32_t zz = z * 0x10001u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t a = t[i >> 1], b = t[2 + (i >> 1)];
        const uint32_t both = __byte_perm(__float_as_uint(i & 1 ? hi32(a) : lo32(a)), __float_as_uint(i & 1 ? hi32(b) : lo32(b)), 0x5410);
        uint32_t d;
        asm("{ .reg .b32 x; add.s16x2 x, %1, %2; min.relu.s16x2 %0, x, %3; }" : "=r"(d) : "r"(both), "r"(zz), "r"(0x000F000Fu));
        c[i] = d;
    }
    bad |= !(s < INFINITY);
    word = (uint32_t)__half_as_ushort(sh) | ((uint32_t)__half_as_ushort(__ushort2half_rn((unsigned short)z)) << 16);
    return s > 0.0f ? (c[0] | c[1] << 4) | (c[2] << 8 | c[3] << 12) : 0u;
}

// A warp's rounds with their rows' places.  Where all R rows lie one after another in
// one sequence (nearly always in a prompt) the places are steps from the first,
// so the addresses are too (fewer instructions: 22.6 -> 20.0 us for 8191 rows in and out).
template <int D, class F>
__device__ __forceinline__ void one_run(const Part<D> &p, long long found, F rounds) {
    const int lane = threadIdx.x & 31;
    const long long first = __shfl_sync(0xffffffffu, found, 0);
    if (first >= 0 && __all_sync(0xffffffffu, lane >= Part<D>::R || found == first + lane)) {
        const long long mine = first + p.g * kRounds;
        rounds([=](int i) { return mine + i; });
    } else {
        rounds([=](int i) { return __shfl_sync(0xffffffffu, found, p.g * kRounds + i); });
    }
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    append_kernel(const uint16_t *__restrict__ k, int ldk, const uint16_t *__restrict__ v, int ldv, Rows r,
                  uint32_t *__restrict__ kc, uint32_t *__restrict__ ks, uint32_t *__restrict__ vc,
                  uint32_t *__restrict__ vs, int32_t *st) {
    constexpr int L = Part<D>::L;
    __shared__ int32_t buf[kStage + 1];
    pdl_launch_dependents();
    const Part<D> p(r);
    pdl_wait();
    check_ranges(r, st);
    uint4 in[2][kRounds];
#pragma unroll
    for (int i = 0; i < kRounds; ++i) {
        const bool there = p.in && p.row(i) < r.rows;
        const size_t m = (size_t)p.row(i);
        in[0][i] = there ? __ldcs(reinterpret_cast<const uint4 *>(k + m * ldk + (size_t)p.hd * D) + p.l) : make_uint4(0, 0, 0, 0);
        in[1][i] = there ? __ldcs(reinterpret_cast<const uint4 *>(v + m * ldv + (size_t)p.hd * D) + p.l) : make_uint4(0, 0, 0, 0);
    }
    const int32_t *start = stage_starts(r, buf);
    if (!p.in) return;
    const long long found = locate<Part<D>::R>(r, start, p.m0, p.hd);
    bool bad = false;
    uint32_t word[2] = {0, 0};                   // of the row that this lane writes
    auto rounds = [&](auto place) {
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const long long at = place(i);
            bool b = false;
            uint32_t kw, vw;
            const uint32_t kn = quantise<L>(in[0][i], kw, b), vn = quantise<L>(in[1][i], vw, b);
            if (at >= 0) {
                kc[at * L + p.l] = kn;
                vc[at * L + p.l] = vn;
                bad |= b;
            }
            if (p.l == i) {
                word[0] = kw;
                word[1] = vw;
            }
        }
    };
    const long long mine = __shfl_sync(0xffffffffu, found, (p.g * kRounds + p.l) & 31);
    one_run<D>(p, found, rounds);
    if (p.l < kRounds && mine >= 0) {            // R words side by side
        ks[mine] = word[0];
        vs[mine] = word[1];
    }
    if (bad) flag(st, QSPEC_ERR_NONFINITE);
}

// 8 codes and a scale word -> 8 bf16 values s (c - z), each rounded once (c - z
// and the product of an fp16 and a 4-bit integer are exact in fp32)
__device__ __forceinline__ uint4 values(uint32_t nib, uint32_t word) {
    const float s = __half2float(__ushort_as_half((uint16_t)(word & 0xFFFFu)));
    const float z = __half2float(__ushort_as_half((uint16_t)(word >> 16)));
    // 2^23 + c by its bits, minus 2^23 + z
    const float zi = -(8388608.0f + z);
    const uint32_t even = nib & 0x0F0F0F0Fu, odd = (nib >> 4) & 0x0F0F0F0Fu;
    uint32_t o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float a = __uint_as_float(__byte_perm(even, 0x4B000000u, 0x7440 | i));
        const float c = __uint_as_float(__byte_perm(odd, 0x4B000000u, 0x7440 | i));
        const uint64_t d = mul2(add2(f2(a, c), f2(zi, zi)), f2(s, s));
        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(hi32(d)), "f"(lo32(d)));
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

template <int D>
__global__ void __launch_bounds__(kThreads)
    load_kernel(const uint32_t *__restrict__ kc, const uint32_t *__restrict__ ks, const uint32_t *__restrict__ vc,
                const uint32_t *__restrict__ vs, Rows r, uint16_t *__restrict__ k, int ldk, uint16_t *__restrict__ v,
                int ldv, int32_t *st) {
    constexpr int L = Part<D>::L;
    __shared__ int32_t buf[kStage + 1];
    pdl_launch_dependents();
    const Part<D> p(r);
    pdl_wait();
    check_ranges(r, st);
    const int32_t *start = stage_starts(r, buf);
    if (!p.in) return;
    const long long found = locate<Part<D>::R>(r, start, p.m0, p.hd);
    auto rounds = [&](auto place) {
        uint32_t kn[kRounds], vn[kRounds], kw[kRounds], vw[kRounds];
        bool there[kRounds];
#pragma unroll
        for (int i = 0; i < kRounds; ++i) {
            const long long at = place(i);
            there[i] = at >= 0;
            kn[i] = there[i] ? __ldg(kc + at * L + p.l) : 0u;
            vn[i] = there[i] ? __ldg(vc + at * L + p.l) : 0u;
            kw[i] = there[i] ? __ldg(ks + at) : 0u;
            vw[i] = there[i] ? __ldg(vs + at) : 0u;
        }
#pragma unroll
        for (int i = 0; i < kRounds; ++i)
            if (there[i]) {
                const size_t m = (size_t)p.row(i);
                reinterpret_cast<uint4 *>(k + m * ldk + (size_t)p.hd * D)[p.l] = values(kn[i], kw[i]);
                reinterpret_cast<uint4 *>(v + m * ldv + (size_t)p.hd * D)[p.l] = values(vn[i], vw[i]);
            }
    };
    one_run<D>(p, found, rounds);
}

// CTAs of a call
template <int D>
long long ctas(long long rows, int H) {
    return ((rows + Part<D>::R - 1) / Part<D>::R * H + kWarps - 1) / kWarps;
}

// what both calls can refuse on the host
int check(const void *k, int ldk, const void *v, int ldv, const int32_t *start, const int32_t *base, int rows, int B,
          int H, int T, int D, const void *kc, const void *ks, const void *vc, const void *vs) {
    if (!start || !base || !kc || !ks || !vc || !vs || (rows > 0 && (!k || !v))) return QSPEC_ERR_NULL;
    if (rows < 0 || rows > INT_MAX - 64 || B < 1 || H < 1 || T < 1 || (D != 64 && D != 128)) return QSPEC_ERR_SHAPE;
    if (ldk < (long long)H * D || ldv < (long long)H * D) return QSPEC_ERR_SHAPE;
    if ((D == 128 ? ctas<128>(rows, H) : ctas<64>(rows, H)) * kWarps >= 1LL << 32) return QSPEC_ERR_SHAPE;
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
    const unsigned grid = (unsigned)(D == 128 ? kv4::ctas<128>(rows, H) : kv4::ctas<64>(rows, H));
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
    const unsigned grid = (unsigned)(D == 128 ? kv4::ctas<128>(rows, H) : kv4::ctas<64>(rows, H));
    auto kern = D == 128 ? kv4::load_kernel<128> : kv4::load_kernel<64>;
    return launch_pdl("qspec_kv4_load", kern, dim3(grid), dim3(kv4::kThreads), 0, as_cuda(stream),
                      reinterpret_cast<const uint32_t *>(k_codes), k_sz, reinterpret_cast<const uint32_t *>(v_codes),
                      v_sz, r, k_bf16, ldk, v_bf16, ldv, dev_status);
}
