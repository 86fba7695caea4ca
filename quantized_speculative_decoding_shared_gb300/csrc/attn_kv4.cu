// attn_kv4.cu -- attention of the newest rows of every sequence over the 4-bit
// KV cache (draft steps and verify passes).
//
//   a_t = scale s_t (sum_d q_d c_td - z_t sum_d q_d),  p = softmax(a),
//   o = sum_t p_t s_t (c_t - z_t)
//
// The R G query rows that read one KV head are taken together, kRows = 8 NT of
// them per pass.  Products run as warp MMAs with the cache on the row side,
// 16 positions by 8 query rows, so that few query rows waste little:
//   S^T (positions x rows) = K Q^T:  a K word's eight codes become four bf16
//     pairs 128 + c by a shift and one logic operation each (the order of d is
//     free: Q is permuted the same way once), and (128 + z) sum q is taken off
//     the fp32 sum;
//   O^T (d x rows) += V^T P^T:  V's codes of two positions side by side, minus
//     (128 + z) exactly in bf16; P^T = p s is S^T's fragment transposed 8 x 8.
// Codes and scale words come through a ring of cp.async stages that each warp
// keeps for itself: no barrier between warps inside a segment.  The
// softmax reference m moves only when a score passes it by more than 2^8.
//
// Work is split by the lengths on the device: all (sequence, head, row block)
// tasks, cut into chunks of 64 positions, are laid end to end and every CTA
// takes an equal share.  A task that several CTAs share is joined by the last
// of them to finish, in the order of the parts, so that the bits do not
// depend on who is last.
//
// Bound: HBM for one row tile (D / 2 + 4 bytes per position, head and side);
// with more rows the warp MMAs and the integer work of unpacking.
#include <algorithm>
#include <cmath>

#include <cuda_fp16.h>

#include "qspec_device.cuh"
#include "qspec_host.h"

namespace qspec {

namespace {

namespace akv {

constexpr int kMaxR = QSPEC_MAX_GAMMA + 1;
constexpr int kWarps = 4, kThreads = kWarps * 32;
constexpr int kTile = 16;                       // positions per MMA tile
constexpr int kChunk = kWarps * kTile;          // positions per unit of work
constexpr int kMaxSms = 160;
constexpr float kNone = -1.0e30f;               // running reference before any score
constexpr float kMove = 8.0f;                   // log2 of the largest p

// CTAs per SM (registers: the O^T accumulators are 4 NT D / 16 per thread)
template <int NT>
constexpr int per_sm() { return NT == 1 ? 4 : NT == 2 ? 3 : 2; }
constexpr int kMaxCtas = kMaxSms * 4;
constexpr int kMaxRowsPerSm = 2 * 32;           // max over NT of per_sm * 8 NT
constexpr int kMaxD = 128;

template <int D>
constexpr int stage_bytes() { return 2 * kTile * (D / 2) + 2 * kTile * 4; }
constexpr int kStages = 6;
template <int D, int NT>
constexpr size_t smem_bytes() {
    // the ring, and over it at the end of a segment the warps' O (rows padded by 4)
    return std::max((size_t)kWarps * kStages * stage_bytes<D>(), (size_t)kWarps * 8 * NT * (D + 4) * 4) +
           (size_t)kWarps * 8 * NT * 2 * 4;
}

struct Args {
    const uint16_t *q;
    const uint8_t *kc, *vc;
    const uint32_t *ks, *vs;
    const int32_t *len;
    uint16_t *o;
    int32_t *st;
    int *count;                                  // [kMaxCtas] arrivals at the task that a CTA begins
    float *part;                                 // partial results, two slots per CTA
    int ldq, ldo, B, R, G, H, T, blocks;         // blocks: row blocks per (sequence, head)
    float scale;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t bf2_sub(uint32_t a, uint32_t b) {
    __nv_bfloat162 r = __hsub2(*reinterpret_cast<__nv_bfloat162 *>(&a), *reinterpret_cast<__nv_bfloat162 *>(&b));
    return *reinterpret_cast<uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t code_pair(uint32_t w, int i) {   // bf16 pair 128 + (nibble i of each half)
    return ((w >> (4 * i)) & 0x000F000Fu) | 0x43004300u;
}
__device__ __forceinline__ float lo_half(uint32_t w) { return __half2float(__ushort_as_half((uint16_t)(w & 0xFFFFu))); }
__device__ __forceinline__ float hi_half(uint32_t w) { return __half2float(__ushort_as_half((uint16_t)(w >> 16))); }
// 128 + z; the clamp keeps a bad word at an unseen place from reaching the
// rows that do not see it as NaN (0 times NaN)
__device__ __forceinline__ float zero_point(uint32_t w) { return 128.0f + fminf(fmaxf(hi_half(w), 0.0f), 15.0f); }

__device__ __forceinline__ void mma(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};\n"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t x) {
    uint32_t y;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
    return y;
}
__device__ __forceinline__ uint32_t saddr(const void *p) { return (uint32_t)__cvta_generic_to_shared(p); }
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, bool in) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(in ? 4 : 0) : "memory");
}

// MMA row of position x (0..15) of a tile: rows 2 i, 2 i + 1, 8 + 2 i, 9 + 2 i are
// positions i, 4 + i, 8 + i, 12 + i, which spreads a thread's V rows over the banks
__device__ __forceinline__ int mma_row(int x) { return (x & 8) | ((x & 3) << 1) | ((x >> 2) & 1); }

template <int D, int NT>
__global__ void __launch_bounds__(kThreads, per_sm<NT>()) attn_kv4_kernel(const __grid_constant__ Args a) {
    constexpr int kRows = 8 * NT;
    constexpr int kWords = D / 32;              // K words per thread and position, V words x 2 ... (D / 64)
    constexpr int kSteps = D / 16;              // MMA steps of S, and 16-row tiles of O^T
    constexpr int kStage = stage_bytes<D>(), kSide = kTile * (D / 2);
    extern __shared__ __align__(16) uint8_t smem[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, g8 = lane >> 2, t4 = lane & 3;
    uint8_t *ring = smem + (size_t)warp * kStages * kStage;
    float *so = reinterpret_cast<float *>(smem);                                   // [warp][row][D + 4]
    float *sml = reinterpret_cast<float *>(smem + smem_bytes<D, NT>()) - kWarps * kRows * 2;   // [warp][row]{m, l}
    __shared__ int last_flag;

    pdl_launch_dependents();
    pdl_wait();
    // ---- this CTA's share of the chunks (every warp finds it for itself) ----
    const int tasks = a.H * a.blocks;           // per sequence
    auto chunks_of = [&](int b) -> int {
        const int n = __ldg(a.len + b);
        return n < 0 || n > a.T ? 0 : max(1, (n + kChunk - 1) / kChunk);
    };
    long long total = 0;
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int c = b0 + lane < a.B ? chunks_of(b0 + lane) : 0;
        if (blockIdx.x == 0 && b0 + lane < a.B && c == 0) flag(a.st, QSPEC_ERR_RANGE);
        total += __reduce_add_sync(0xffffffffu, c);
    }
    total *= tasks;
    const long long nc = min((long long)gridDim.x, total);
    if (blockIdx.x >= nc) return;
    long long at = blockIdx.x * total / nc;
    const long long end = (blockIdx.x + 1) * total / nc;
    int b = 0;
    long long prefix = 0;                        // items before sequence b
    for (int b0 = 0; b0 < a.B; b0 += 32) {
        const int c = b0 + lane < a.B ? chunks_of(b0 + lane) : 0;
        int upto = c;
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, upto, x);
            if (lane >= x) upto += y;
        }
        const uint32_t past = __ballot_sync(0xffffffffu, prefix + (long long)upto * tasks > at);
        if (past) {
            const int who = __ffs(past) - 1;
            b = b0 + who;
            prefix += (long long)(__shfl_sync(0xffffffffu, upto, who) - __shfl_sync(0xffffffffu, c, who)) * tasks;
            break;
        }
        prefix += (long long)__shfl_sync(0xffffffffu, upto, 31) * tasks;
    }
    int chunks = chunks_of(b);
    int task = (int)((at - prefix) / chunks), chunk = (int)((at - prefix) - (long long)task * chunks);

    while (at < end) {
        // ---- one segment: chunks [chunk, chunk + n_ch) of a task ----
        const int n_ch = (int)min((long long)(chunks - chunk), end - at);
        const int len = __ldg(a.len + b), h = task / a.blocks, row0 = (task - h * a.blocks) * kRows;
        const int nq = min(kRows, a.R * a.G - row0);
        const int p0 = chunk * kChunk, p1 = min(len, p0 + n_ch * kChunk);
        const size_t head = ((size_t)b * a.H + h) * a.T;
        const int tiles = max(0, (p1 - p0 + kTile - 1) / kTile);
        auto issue = [&](int i, int stage) {                         // this warp's tile i: positions p0 + 16 (4 i + warp)
            const int pt = p0 + kTile * (kWarps * i + warp);
            if (pt < p1) {
                const uint32_t dst = saddr(ring + stage * kStage);
                constexpr int kPer = D / 32;                          // 16-byte pieces per position
#pragma unroll
                for (int e = 0; e < kTile * kPer / 32; ++e) {
                    const int x = (e * 32 + lane) / kPer, c = (e * 32 + lane) % kPer;
                    const bool in = pt + x < p1;
                    const size_t src = (head + (in ? pt + x : p0)) * (D / 2) + 16 * c;
                    copy16(dst + mma_row(x) * (D / 2) + 16 * c, a.kc + src, in);
                    copy16(dst + kSide + x * (D / 2) + 16 * (D == 128 ? c ^ (x & 2) : c), a.vc + src, in);
                }
                const int x = lane & 15;
                const bool in = pt + x < p1;
                copy4(dst + 2 * kSide + (lane & 16) * 4 + mma_row(x) * 4, (lane < 16 ? a.ks : a.vs) + head + (in ? pt + x : p0),
                      in);
            }
            asm volatile("cp.async.commit_group;" ::: "memory");
        };
        const int mine = (tiles - warp + kWarps - 1) / kWarps;       // tiles of this warp (0 or fewer: none)
#pragma unroll
        for (int s = 0; s < kStages - 1; ++s) issue(s, s);

        // ---- Q fragments (k order: pairs (i, i + 4) of a word's eight d) and sum q ----
        uint32_t qf[NT][kSteps][2];
        float qs[NT][2];
#pragma unroll
        for (int j = 0; j < NT; ++j) {
            const int n = row0 + 8 * j + g8, r = n / a.G, gg = n - r * a.G;
            float sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWords; ++w) {
                uint4 x = make_uint4(0, 0, 0, 0);
                if (8 * j + g8 < nq)
                    x = __ldg(reinterpret_cast<const uint4 *>(a.q + (size_t)(b * a.R + r) * a.ldq + (size_t)(h * a.G + gg) * D +
                                                              (D / 4) * t4 + 8 * w));
                const uint32_t v[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) sum += __uint_as_float(v[e] << 16) + __uint_as_float(v[e] & 0xFFFF0000u);
                qf[j][2 * w][0] = __byte_perm(x.x, x.z, 0x5410);
                qf[j][2 * w][1] = __byte_perm(x.x, x.z, 0x7632);
                qf[j][2 * w + 1][0] = __byte_perm(x.y, x.w, 0x5410);
                qf[j][2 * w + 1][1] = __byte_perm(x.y, x.w, 0x7632);
            }
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            qs[j][0] = __shfl_sync(0xffffffffu, sum, 8 * t4);        // rows 2 t, 2 t + 1: the S^T columns of this thread
            qs[j][1] = __shfl_sync(0xffffffffu, sum, 8 * t4 + 4);
        }
        const float cs = a.scale * 1.4426950408889634f;
        float m[NT][2], l[NT][2], acc[kSteps][NT][4];
        int seen[NT][2];                                              // positions that a row sees
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                m[j][e] = kNone;
                l[j][e] = 0.0f;
                seen[j][e] = len - a.R + 1 + (row0 + 8 * j + 2 * t4 + e) / a.G;
            }
#pragma unroll
        for (int i = 0; i < kSteps; ++i)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[i][j][e] = 0.0f;

        for (int i = 0; i < mine; ++i) {
            asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 2) : "memory");
            __syncwarp();
            issue(i + kStages - 1, (i + kStages - 1) % kStages);
            const uint8_t *stg = ring + (i % kStages) * kStage;
            const uint32_t *szk = reinterpret_cast<const uint32_t *>(stg + 2 * kSide), *szv = szk + kTile;
            // ---- S^T = K Q^T ----
            float s[NT][4];
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) s[j][e] = 0.0f;
            uint32_t kw[2][kWords];
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const uint8_t *src = stg + (g8 + 8 * e) * (D / 2) + t4 * (D / 8);
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(src);
                    kw[e][0] = x.x, kw[e][1] = x.y, kw[e][2] = x.z, kw[e][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(src);
                    kw[e][0] = x.x, kw[e][1] = x.y;
                }
            }
#pragma unroll
            for (int k = 0; k < kSteps; ++k) {
                const int w = k >> 1, f = 2 * (k & 1);
                const uint32_t a0 = code_pair(kw[0][w], f), a1 = code_pair(kw[1][w], f), a2 = code_pair(kw[0][w], f + 1),
                               a3 = code_pair(kw[1][w], f + 1);
#pragma unroll
                for (int j = 0; j < NT; ++j) mma(s[j], a0, a1, a2, a3, qf[j][k][0], qf[j][k][1]);
            }
            const uint32_t k0w = szk[g8], k1w = szk[g8 + 8];
            const float sk[2] = {lo_half(k0w) * cs, lo_half(k1w) * cs}, zk[2] = {128.0f + hi_half(k0w), 128.0f + hi_half(k1w)};
            // scores in log2 units; places that a row does not see
            const int pt = p0 + kTile * (kWarps * i + warp);
            const bool edge = pt + kTile > len - a.R + 1;
            const int pos = pt + ((g8 & 1) << 2) + (g8 >> 1);         // position of MMA row g8 (row g8 + 8: + 8)
            bool move = false;
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    s[j][e] = sk[e >> 1] * fmaf(-zk[e >> 1], qs[j][e & 1], s[j][e]);
                    if (edge && pos + 8 * (e >> 1) >= seen[j][e & 1]) s[j][e] = -INFINITY;
                    move |= s[j][e] > m[j][e & 1] + kMove;
                }
            if (__any_sync(0xffffffffu, move)) {
#pragma unroll
                for (int j = 0; j < NT; ++j)
#pragma unroll
                    for (int e = 0; e < 2; ++e) {
                        float top = fmaxf(s[j][e], s[j][e + 2]);
#pragma unroll
                        for (int x = 4; x <= 16; x <<= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                        if (top > m[j][e] + kMove) {
                            const float f = ex2(m[j][e] - top);
                            m[j][e] = top;
                            l[j][e] *= f;
#pragma unroll
                            for (int k = 0; k < kSteps; ++k) {
                                acc[k][j][e] *= f;
                                acc[k][j][e + 2] *= f;
                            }
                        }
                    }
            }
            // ---- p, l, and P^T fragments ----
            const float v0 = lo_half(szv[g8]), v1 = lo_half(szv[g8 + 8]);
            uint32_t pf[NT][2];
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                float p[4];
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    p[e] = ex2(s[j][e] - m[j][e & 1]);
                    l[j][e & 1] += p[e];
                }
                float w[4] = {p[0] * v0, p[1] * v0, p[2] * v1, p[3] * v1};
                if (edge)                                             // an unseen place's scale may be anything
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[e] = p[e] == 0.0f ? 0.0f : w[e];
                pf[j][0] = transpose8x8(pack_bf16(w[0], w[1]));
                pf[j][1] = transpose8x8(pack_bf16(w[2], w[3]));
            }
            // ---- O^T += V^T P^T: MMA rows 2 t, 2 t + 1 and 8 + 2 t, 9 + 2 t of the tile ----
            const uint2 za = *reinterpret_cast<const uint2 *>(szv + 2 * t4), zb = *reinterpret_cast<const uint2 *>(szv + 8 + 2 * t4);
            const uint32_t zz0 = pack_bf16(zero_point(za.x), zero_point(za.y)), zz1 = pack_bf16(zero_point(zb.x), zero_point(zb.y));
            const uint8_t *vsrc = stg + kSide + t4 * (D / 2) + (D == 128 ? ((8 * g8) ^ ((t4 & 2) << 4)) : 4 * g8);
            uint32_t vw[4][D / 64];
#pragma unroll
            for (int x = 0; x < 4; ++x) {                             // positions t, 4 + t, 8 + t, 12 + t
                if constexpr (D == 128) {
                    const uint2 y = *reinterpret_cast<const uint2 *>(vsrc + x * 4 * (D / 2));
                    vw[x][0] = y.x, vw[x][1] = y.y;
                } else {
                    vw[x][0] = *reinterpret_cast<const uint32_t *>(vsrc + x * 4 * (D / 2));
                }
            }
#pragma unroll
            for (int w = 0; w < D / 64; ++w) {
                const uint32_t l0 = __byte_perm(vw[0][w], vw[1][w], 0x5410), h0 = __byte_perm(vw[0][w], vw[1][w], 0x7632),
                               l1 = __byte_perm(vw[2][w], vw[3][w], 0x5410), h1 = __byte_perm(vw[2][w], vw[3][w], 0x7632);
#pragma unroll
                for (int f = 0; f < 4; ++f) {
                    const uint32_t a0 = bf2_sub(code_pair(l0, f), zz0), a1 = bf2_sub(code_pair(h0, f), zz0),
                                   a2 = bf2_sub(code_pair(l1, f), zz1), a3 = bf2_sub(code_pair(h1, f), zz1);
#pragma unroll
                    for (int j = 0; j < NT; ++j) mma(acc[4 * w + f][j], a0, a1, a2, a3, pf[j][0], pf[j][1]);
                }
            }
        }
        asm volatile("cp.async.wait_group 0;" ::: "memory");

        // ---- the warps' results joined: rows 2 t, 2 t + 1 of each 8, d = (D / 8) g + ... ----
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
#pragma unroll
                for (int x = 4; x <= 16; x <<= 1) l[j][e] += __shfl_xor_sync(0xffffffffu, l[j][e], x);
                if (g8 == 0)
                    *reinterpret_cast<float2 *>(sml + (warp * kRows + 8 * j + 2 * t4 + e) * 2) = make_float2(m[j][e], l[j][e]);
            }
        __syncthreads();                                              // every warp is done with its ring
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int e = 0; e < 2; ++e) {
                const int n = 8 * j + 2 * t4 + e;
                float top = kNone;
#pragma unroll
                for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sml[(w * kRows + n) * 2]);
                const float f = ex2(m[j][e] - top);
                float *dst = so + (size_t)(warp * kRows + n) * (D + 4) + (D / 8) * g8;
#pragma unroll
                for (int w = 0; w < D / 64; ++w) {                    // word w: d 0..3 in MMA row g, 4..7 in row g + 8
                    *reinterpret_cast<float4 *>(dst + 8 * w) = make_float4(acc[4 * w][j][e] * f, acc[4 * w + 1][j][e] * f,
                                                                           acc[4 * w + 2][j][e] * f, acc[4 * w + 3][j][e] * f);
                    *reinterpret_cast<float4 *>(dst + 8 * w + 4) =
                        make_float4(acc[4 * w][j][e + 2] * f, acc[4 * w + 1][j][e + 2] * f, acc[4 * w + 2][j][e + 2] * f,
                                    acc[4 * w + 3][j][e + 2] * f);
                }
            }
        __syncthreads();
        const long long ts = prefix + (long long)task * chunks;       // the task's first item
        const bool whole = n_ch == chunks;
        const int c0 = (int)(((ts + 1) * nc + total - 1) / total) - 1, c1 = (int)(((ts + chunks) * nc + total - 1) / total) - 1;
        constexpr int kSlot = kRows * (D + 2);
        auto out_row = [&](int n) {
            const int r = (row0 + n) / a.G, gg = (row0 + n) - r * a.G;
            return a.o + (size_t)(b * a.R + r) * a.ldo + (size_t)(h * a.G + gg) * D;
        };
        float *slot = a.part + ((size_t)blockIdx.x * 2 + ((int)blockIdx.x == c0 ? 1 : 0)) * kSlot;
        for (int n = warp; n < nq; n += kWarps) {                      // a warp per row, four d per lane
            float top = kNone, sum = 0.0f;
#pragma unroll
            for (int w = 0; w < kWarps; ++w) top = fmaxf(top, sml[(w * kRows + n) * 2]);
#pragma unroll
            for (int w = 0; w < kWarps; ++w) sum += sml[(w * kRows + n) * 2 + 1] * ex2(sml[(w * kRows + n) * 2] - top);
            if (4 * lane < D) {
                float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
                for (int w = 0; w < kWarps; ++w) {
                    const float4 y = *reinterpret_cast<const float4 *>(so + (size_t)(w * kRows + n) * (D + 4) + 4 * lane);
                    x.x += y.x, x.y += y.y, x.z += y.z, x.w += y.w;
                }
                if (whole) {
                    const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;   // NaN stays
                    *reinterpret_cast<uint2 *>(out_row(n) + 4 * lane) =
                        make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
                } else {
                    __stcg(reinterpret_cast<float4 *>(slot + n * D + 4 * lane), x);
                }
            }
            if (!whole && lane == 0) __stcg(reinterpret_cast<float2 *>(slot + kRows * D + 2 * n), make_float2(top, sum));
        }
        if (!whole) {
            __syncthreads();
            if (tid == 0) {
                __threadfence();
                const int done = atomicAdd(a.count + c0, 1);
                last_flag = done == c1 - c0;
                if (last_flag) {
                    a.count[c0] = 0;                                   // ready for the next call
                    __threadfence();
                }
            }
            __syncthreads();
            if (last_flag) {
                auto part = [&](int c) { return a.part + ((size_t)c * 2 + (c == c0 ? 1 : 0)) * kSlot; };
                for (int n = warp; n < nq; n += kWarps) {
                    float top = kNone;
                    for (int c = c0 + lane; c <= c1; c += 32) top = fmaxf(top, __ldcg(part(c) + kRows * D + 2 * n));
#pragma unroll
                    for (int x = 16; x >= 1; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
                    float sum = 0.0f;
                    float4 x = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                    for (int cb = c0; cb <= c1; cb += 32) {
                        float2 ml = make_float2(kNone, 0.0f);
                        if (cb + lane <= c1) ml = __ldcg(reinterpret_cast<const float2 *>(part(cb + lane) + kRows * D + 2 * n));
                        const float f = ex2(ml.x - top);
                        const int cnt = min(32, c1 - cb + 1);
#pragma unroll 8
                        for (int c = 0; c < cnt; ++c) {
                            const float fc = __shfl_sync(0xffffffffu, f, c);
                            sum = fmaf(fc, __shfl_sync(0xffffffffu, ml.y, c), sum);
                            if (4 * lane < D) {
                                const float4 y = __ldcg(reinterpret_cast<const float4 *>(part(cb + c) + n * D + 4 * lane));
                                x.x = fmaf(fc, y.x, x.x), x.y = fmaf(fc, y.y, x.y), x.z = fmaf(fc, y.z, x.z), x.w = fmaf(fc, y.w, x.w);
                            }
                        }
                    }
                    const float inv = sum > 0.0f ? 1.0f / sum : sum == 0.0f ? 0.0f : sum;
                    if (4 * lane < D)
                        *reinterpret_cast<uint2 *>(out_row(n) + 4 * lane) =
                            make_uint2(pack_bf16(x.x * inv, x.y * inv), pack_bf16(x.z * inv, x.w * inv));
                }
            }
        }
        __syncthreads();                                              // shared memory free for the next segment
        // ---- on to the next task ----
        at += n_ch;
        chunk = 0;
        if (++task == tasks && at < end) {
            task = 0;
            prefix += (long long)chunks * tasks;
            do chunks = chunks_of(++b);
            while (chunks == 0);
        }
    }
}

bool sizes_ok(int B, int R, int Hq, int H, int D) {
    return B >= 1 && R >= 1 && R <= kMaxR && H >= 1 && Hq >= H && Hq % H == 0 && (D == 64 || D == 128) &&
           (long long)B * R * Hq < (1LL << 28);
}

constexpr size_t kCountBytes = kMaxCtas * sizeof(int);

template <int D, int NT>
int launch(Args a, cudaStream_t stream) {
    a.blocks = (a.R * a.G + 8 * NT - 1) / (8 * NT);
    auto kern = attn_kv4_kernel<D, NT>;
    int rc = smem_limit_once(reinterpret_cast<const void *>(kern), (int)smem_bytes<D, NT>(), true);
    if (rc) return rc;
    const long long most = (long long)a.B * a.H * a.blocks * std::max(1, (a.T + kChunk - 1) / kChunk);   // chunks at full lengths
    const unsigned grid = (unsigned)std::min<long long>((long long)std::min(sm_count(), kMaxSms) * per_sm<NT>(), most);
    return launch_pdl("qspec_attn_kv4", kern, dim3(grid), dim3(kThreads), smem_bytes<D, NT>(), stream, a);
}

// row tiles per pass: the fewest passes over the cache with at most four, evenly filled
template <int D>
int dispatch(const Args &a, cudaStream_t stream) {
    const int tiles = (a.R * a.G + 7) / 8, passes = (tiles + 3) / 4;
    switch ((tiles + passes - 1) / passes) {
        case 1: return launch<D, 1>(a, stream);
        case 2: return launch<D, 2>(a, stream);
        case 3: return launch<D, 3>(a, stream);
        default: return launch<D, 4>(a, stream);
    }
}

}  // namespace akv

}  // namespace

}  // namespace qspec

using namespace qspec;

extern "C" size_t qspec_attn_kv4_workspace_bytes(int B, int R, int Hq, int H, int D) {
    // the same for every shape: arrival counts, then the partial results of every CTA that can be resident
    return akv::sizes_ok(B, R, Hq, H, D)
               ? akv::kCountBytes + (size_t)akv::kMaxSms * akv::kMaxRowsPerSm * 2 * (akv::kMaxD + 2) * sizeof(float)
               : 0;
}

extern "C" int qspec_attn_kv4(const uint16_t *q_bf16, int ldq, const uint8_t *k_codes, const uint32_t *k_sz,
                              const uint8_t *v_codes, const uint32_t *v_sz, const int32_t *len, int B, int R, int Hq,
                              int H, int T, int D, float scale, uint16_t *o_bf16, int ldo, void *workspace,
                              size_t ws_bytes, int32_t *dev_status, qspec_stream_t stream) {
    if (!q_bf16 || !k_codes || !k_sz || !v_codes || !v_sz || !len || !o_bf16 || !workspace) return QSPEC_ERR_NULL;
    if (!akv::sizes_ok(B, R, Hq, H, D) || T < 1 || T > (1 << 30) || !std::isfinite(scale) || ldq < (long long)Hq * D ||
        ldo < (long long)Hq * D)
        return QSPEC_ERR_SHAPE;
    if (ldq % 8 || ldo % 8 || !aligned(q_bf16, 16) || !aligned(o_bf16, 16) || !aligned(k_codes, 16) ||
        !aligned(v_codes, 16) || !aligned(k_sz, 4) || !aligned(v_sz, 4) || !aligned(len, 4) || !aligned(workspace, 16))
        return QSPEC_ERR_ALIGN;
    if (ws_bytes < qspec_attn_kv4_workspace_bytes(B, R, Hq, H, D)) return QSPEC_ERR_WORKSPACE;
    int rc = check_device();
    if (rc) return rc;
    const akv::Args a{q_bf16, k_codes, v_codes, k_sz, v_sz, len, o_bf16, dev_status, reinterpret_cast<int *>(workspace),
                      reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + akv::kCountBytes), ldq, ldo, B, R,
                      Hq / H, H, T, 1, scale};
    return D == 128 ? akv::dispatch<128>(a, as_cuda(stream)) : akv::dispatch<64>(a, as_cuda(stream));
}
