// attn_kv4.cu -- attention of the newest rows of every sequence over the 4-bit
// KV cache (draft steps and verify passes), on the Blackwell tensor cores.
//
//   a_t = scale s_t (sum_d q_d c_td - z_t sum_d q_d),  p = softmax(a),
//   o = sum_t p_t s_t (c_t - z_t)
//
// The R G query rows that read one KV head are taken together, N (16, 32 or 64)
// of them per pass, as the narrow side of the products; 128 cache positions are
// the wide one:
//   S^T (positions x rows) = K Q^T in fp16: a code c in the low bits of an fp16
//     lane IS the number c 2^-24 (a subnormal), one nibble higher 16 c 2^-24, so eight
//     codes take one shift and four ANDs on their way into tensor memory (thread
//     = position).  Each row of Q is scaled by a power of two to at most 2^15
//     (exact: bf16 has 8 bits, fp16 11, and what falls below 2^-24 is below 2^-39
//     of the row's largest), in the order of d that the unpacked codes have, times 1/16
//     against 16 c.  z enters as one more K step: z against -sum q in three fp16 parts.
//   O^T (d x rows) += V^T P^T in bf16: c - z exactly; P^T = p s with the range of fp32 (in fp16 the weights of
//     far positions would round to subnormals).  Both operands lie in shared memory
//     position by position, an MN-major layout without swizzle: 16-byte pieces of
//     consecutive positions side by side.
// Three groups of four warps take the tiles in turn (thread = position: unpack K,
// unpack V while S^T is formed, then the softmax); one lane issues the products of
// S^T, one those of O^T (each waits for its own operands, so that the tensor cores
// have the other's meanwhile: at these widths a product takes some 55 clocks
// whatever N is, 17 of them a tile), one the copies, and one tells other CTAs of
// finished parts.
//
// The softmax reference of a row is its score at the segment's first position, and stays:
// p, its sum and O are floating point and lose nothing while no score passes
// it by 2^96.  A segment where one does is taken again by a plain path (a warp to a row, key by
// key: 4 sequences of 8192, one row of 4 heads 0.75 ms for 0.022).  Weights below 2^-126 of the reference are 0.
//
// Work is split by the lengths on the device: all (sequence, head, row block)
// tasks, cut into tiles of 128 positions, are laid end to end, each with a few
// empty tiles in front that stand for a segment's fixed cost (or cut into parts of
// their own, where there is a CTA for each), and every CTA
// takes an equal share.  A task that several CTAs share is joined by the last
// of them to finish, in the order of the parts, so that the bits do not
// depend on who is last.
//
// Bound: the 17 products of a tile (935 of some 1170 clocks at 16 rows) and shared
// memory (half its rate: codes in, V and P^T out and read by the products), HBM next:
// 4 sequences of up to 65001 positions (232840 together), 8 KV heads of 128, one row of 4 heads: 59.2 us, 4.3
// TB/s of the D / 2 + 4 bytes per position, head and side (37.4 us at HBM's rate).  With
// warp MMA (registers only) it was 63.5 us, and 43 for 20.7 at 16 sequences of up to
// 4091 with 5 rows; 32 sequences, 9 rows, 7 heads to a KV head: 29.8 us.  Short calls
// are the way through one tile: 6.3 us for one sequence of 333.
#include <algorithm>
#include <cmath>
#include <type_traits>

#include <cuda_fp16.h>

#include "qspec_device.cuh"
#include "qspec_host.h"
#include "umma.cuh"

namespace qspec {

namespace {

namespace akv {

constexpr int kMaxR = QSPEC_MAX_GAMMA + 1;
constexpr int kTok = 128;                       // positions per tile
template <int N>
struct Cfg {
    static constexpr int kGroups = 3, kWorkWarps = 4 * kGroups, kWork = 32 * kWorkWarps;
    static constexpr int kScoreWarp = kWorkWarps, kValueWarp = kScoreWarp + 1, kLoadWarp = kValueWarp + 1, kTellWarp = kLoadWarp + 1;   // one lane each: S^T, O^T products, copies, finished parts
    static constexpr int kThreads = kWork + 128;
    // registers per thread: all start with 128 and share what that makes (with 128 for the working warps 64 rows
    // spill their sums: 40.1 for 32.1 us at 32 sequences, 9 rows, 7 heads)
    static constexpr int kRegsWork = 144, kRegsRest = 64;
    static_assert(kThreads * 128 <= 65536 && kWork * kRegsWork + 128 * kRegsRest <= kThreads * 128, "register shares");
    // Tiles of codes in flight.  A stage always serves the same group: one whose next tile came into another
    // group's stage could look at that stage's barrier a whole phase early, and take the phase before for its own.
    static constexpr int kStages = N == 16 ? 6 : 3;
    static_assert(kStages % kGroups == 0, "a stage serves one group");
};
constexpr int kMaxCtas = 160;                   // one per SM
constexpr int kMaxN = 64, kMaxD = 128;
constexpr float kNone = -1.0e30f;               // log2 of the sum of a row that sees nothing
constexpr float kOver = 7.9228162514264338e28f; // 2^96: a thread's sum of p from where a segment is taken again

constexpr int kMaxStages = 6;
constexpr int kVBuf = kTok * kMaxD * 2;         // V operand (D = 64: the products' rows 64 .. 127 read the rest, unused)
template <int D>
constexpr int side_bytes() { return kTok * D / 2; }
template <int N>
constexpr int p_bytes() { return kTok * N * 2; }
template <int D, int N>
constexpr int q_bytes() { return N * (D + 16) * 2; }

struct Join {                                   // a task to join: its parts (0: nothing to do)
    int parts, c0, nq, b, task;
};

template <int N>
struct Ctl {
    static constexpr int kGroups = Cfg<N>::kGroups, kWorkWarps = Cfg<N>::kWorkWarps;
    uint64_t full[kMaxStages], empty[kMaxStages];     // codes landed; unpacked
    uint64_t kfull[kGroups], sfull[kGroups], pfull[kGroups], vfull[kGroups], pdone[kGroups];   // K in tensor memory, S^T, P^T, V, O^T += done
    uint64_t qfull, ref, odone, drain[2];       // per segment: Q written, reference known, O^T complete
    uint64_t stored[2];                         // once: results of the part of a task that the CTA continues, begins
    float4 back[N / 2];                         // score of rows n, n + 1: {back, back'}({s u - ref, s u' - ref'}), as {back, back', -ref, -ref'}
    alignas(16) float lse[N], inv[N];
    float lsum[kWorkWarps][N];
    long long orow[N];                          // the rows' places in q and o
    int seen[N];                                // positions that a row sees
    uint32_t tmem;
    int timeout, over;
    Join join[2];                               // the task that the CTA continues, the one that it begins
};

template <int D, int N>
constexpr size_t smem_bytes() {
    return 1024 + (size_t)Cfg<N>::kStages * 2 * side_bytes<D>() + Cfg<N>::kGroups * (kVBuf + p_bytes<N>()) + q_bytes<D, N>() + sizeof(Ctl<N>);
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
    uint32_t g_mul;                              // n / G = umulhi(n, g_mul) for n < 17 G (G = 1: 0)
    float scale;

    __device__ __forceinline__ int row_r(int n) const { return g_mul ? (int)__umulhi((uint32_t)n, g_mul) : n; }
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
__device__ __forceinline__ uint32_t pack_half(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}
// two fp32 values in a register pair, and the packed operations on them
__device__ __forceinline__ uint64_t f2(float a, float b) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ float lo32(uint64_t v) { return __uint_as_float((uint32_t)v); }
__device__ __forceinline__ float hi32(uint64_t v) { return __uint_as_float((uint32_t)(v >> 32)); }
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
__device__ __forceinline__ float lo_half(uint32_t w) { return __half2float(__ushort_as_half((uint16_t)(w & 0xFFFFu))); }
__device__ __forceinline__ float hi_half(uint32_t w) { return __half2float(__ushort_as_half((uint16_t)(w >> 16))); }

__device__ __forceinline__ void bar_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
// the 16-byte piece c of position t in a tile of codes as the copy left it: rows of 64 bytes in
// the 64-byte swizzle, rows of 32 bytes in the 32-byte one
template <int D>
__device__ __forceinline__ uint4 code_piece(const uint8_t *side, int t, int c) {
    if constexpr (D == 128) return *reinterpret_cast<const uint4 *>(side + t * 64 + ((c ^ ((t >> 1) & 3)) << 4));
    return *reinterpret_cast<const uint4 *>(side + t * 32 + ((c ^ ((t >> 2) & 1)) << 4));
}
// d of place x of an operand's piece of eight: the order that unpacking gives
__device__ __forceinline__ int place_d(int x) { return (x >> 1) | ((x & 1) << 2); }

// Sums over the warp's lanes of v[0 .. N - 1]: lane i gets the sum of v[(N / 32) i ..] (N / 32
// values), or for N = 16 of v[i / 2].  Each exchange halves the values a lane still carries.
template <int N>
__device__ __forceinline__ void lane_sums(float (&v)[N], int lane) {
    constexpr int kLast = N >= 32 ? N / 32 : 1;
#pragma unroll
    for (int o = 16, k = N; o >= 1; o >>= 1) {
        if (k > kLast) {
            k >>= 1;
#pragma unroll
            for (int i = 0; i < N / 2; ++i)
                if (i < k) {
                    const bool up = lane & o;
                    const float give = up ? v[i] : v[i + k], keep = up ? v[i + k] : v[i];
                    v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
                }
        } else {
#pragma unroll
            for (int i = 0; i < kLast; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
        }
    }
}

// A row over positions [p0, p1) in the plain order by one warp; o normalised.  Returns log2 of
// the sum of exponentials.
template <int D>
__device__ __noinline__ float plain_row(const Args &a, const uint16_t *qrow, size_t head, int p0, int p1, float (&o)[D / 32]) {
    constexpr int E = D / 32;
    const int lane = threadIdx.x & 31;
    float qv[E], m = -INFINITY, l = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qv[e] = bf16_bits_to_float(qrow[lane * E + e]);
        o[e] = 0.0f;
    }
    for (int t = p0; t < p1; ++t) {
        const uint32_t kw = __ldg(a.ks + head + t), vw = __ldg(a.vs + head + t);
        const float ks = lo_half(kw), kz = hi_half(kw), vs = lo_half(vw), vz = hi_half(vw);
        float s = 0.0f, v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            const int d = lane * E + e, sh = 4 * (d & 1);
            const size_t at = (head + t) * (D / 2) + d / 2;
            s = fmaf(qv[e], (float)((a.kc[at] >> sh) & 15) - kz, s);
            v[e] = vs * ((float)((a.vc[at] >> sh) & 15) - vz);
        }
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
        s *= ks * a.scale * 1.4426950408889634f;
        const float m1 = fmaxf(m, s), ref = m1 > -INFINITY ? m1 : 0.0f, f = ex2(m - ref), p = ex2(s - ref);
        m = m1;
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < E; ++e) o[e] = fmaf(p, v[e], o[e] * f);
    }
    if (l == 0.0f) return kNone;
#pragma unroll
    for (int e = 0; e < E; ++e) o[e] /= l;
    return m + log2f(l);
}

template <int D, int N>
__global__ void __launch_bounds__(Cfg<N>::kThreads, 1)
    attn_kv4_kernel(const __grid_constant__ CUtensorMap tk, const __grid_constant__ CUtensorMap tv,
                    const __grid_constant__ Args a, uint32_t wait_limit, int stall) {
    constexpr int kSide = side_bytes<D>(), kP = p_bytes<N>(), kStages = Cfg<N>::kStages;
    constexpr int kGroups = Cfg<N>::kGroups, kWorkWarps = Cfg<N>::kWorkWarps, kWork = Cfg<N>::kWork;
    constexpr int kScoreWarp = Cfg<N>::kScoreWarp, kValueWarp = Cfg<N>::kValueWarp, kLoadWarp = Cfg<N>::kLoadWarp, kTellWarp = Cfg<N>::kTellWarp;
    constexpr int kSteps = D / 16;                               // MMA steps of S^T (one more holds z)
    constexpr uint32_t cS = 0, cK = kGroups * N, cO = cK + kGroups * 80;   // the groups' S^T and K operands (80 columns each), O^T
    constexpr uint32_t kCols = 512;
    static_assert(cO + N <= kCols, "tensor memory");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    // (an offset, not a rounded address: the compiler keeps seeing shared memory)
    uint8_t *codes = smem_raw + ((1024u - (umma::smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *sv = codes + kStages * 2 * kSide, *sp = sv + kGroups * kVBuf, *sq = sp + kGroups * kP;
    Ctl<N> &sm = *reinterpret_cast<Ctl<N> *>(sq + q_bytes<D, N>());
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

    if (warp == kScoreWarp) umma::tmem_alloc(&sm.tmem, kCols);
    if (tid == 0) {
        for (int s = 0; s < kStages; ++s) {
            umma::mbar_init(&sm.full[s], 1);
            umma::mbar_init(&sm.empty[s], 4);
        }
        for (int s = 0; s < kGroups; ++s) {
            umma::mbar_init(&sm.kfull[s], 4);
            umma::mbar_init(&sm.sfull[s], 1);
            umma::mbar_init(&sm.pfull[s], 4);
            umma::mbar_init(&sm.vfull[s], 4);
            umma::mbar_init(&sm.pdone[s], 1);
        }
        umma::mbar_init(&sm.qfull, kWorkWarps);
        umma::mbar_init(&sm.ref, 1);
        umma::mbar_init(&sm.odone, 1);
        umma::mbar_init(&sm.stored[0], kWorkWarps);
        umma::mbar_init(&sm.stored[1], kWorkWarps);
        umma::mbar_init(&sm.drain[0], 1);
        umma::mbar_init(&sm.drain[1], 1);
        sm.timeout = 0;
        sm.over = 0;
        sm.join[0].parts = sm.join[1].parts = 0;
        umma::mbar_fence_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    const int my_len = lane < a.B ? __ldg(a.len + lane) : -1;    // the first 32 sequences', kept (asked for before the barrier)
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = sm.tmem;
    // A wait that runs out is remembered; from then on no wait waits and nothing
    // more is issued, and every warp walks to the end past the same barriers.
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (umma::mbar_try_wait(bar, parity & 1)) return true;
        if (*reinterpret_cast<volatile int *>(&sm.timeout)) return false;
        if (umma::mbar_wait(bar, parity & 1, wait_limit)) return true;
        *reinterpret_cast<volatile int *>(&sm.timeout) = 1;
        return false;
    };

    // (the votes keep an issuing warp together where a wait runs out)
    auto all = [](bool mine) { return __all_sync(0xffffffffu, mine) != 0; };

    // ---- this CTA's share of the tiles (every warp finds it for itself; 32-bit numbers, the host sees to it: with
    // 64-bit divisions this took 2 us) ----
    const int tasks = a.H * a.blocks;           // per sequence
    auto tiles_in = [&](int n) { return n < 0 || n > a.T ? 0 : max(1, (n + kTok - 1) / kTok); };
    auto tiles_of = [&](int b) { return tiles_in(__ldg(a.len + b)); };
    auto scan = [&](int c) {                    // inclusive, over the lanes
#pragma unroll
        for (int x = 1; x < 32; x <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, c, x);
            if (lane >= x) c += y;
        }
        return c;
    };
    const int mine = tiles_in(my_len), mine_upto = scan(mine);
    auto len_of = [&](int b) { return b < 32 ? __shfl_sync(0xffffffffu, my_len, b) : __ldg(a.len + b); };
    if (blockIdx.x == 0 && warp == 0 && lane < a.B && mine == 0) flag(a.st, QSPEC_ERR_RANGE);
    int total = __shfl_sync(0xffffffffu, mine_upto, 31), valid = __popc(__ballot_sync(0xffffffffu, mine > 0));   // tiles; sequences with tasks
    for (int b0 = 32; b0 < a.B; b0 += 32) {
        const int c = b0 + lane < a.B ? tiles_of(b0 + lane) : 0;
        if (blockIdx.x == 0 && warp == 0 && b0 + lane < a.B && c == 0) flag(a.st, QSPEC_ERR_RANGE);
        total += __reduce_add_sync(0xffffffffu, c);
        valid += __popc(__ballot_sync(0xffffffffu, c > 0));
    }
    total *= tasks;
    const int each = valid * tasks;             // tasks in all
    // Beginning and ending a segment (Q, the first tile's way through the products, sums, results) takes as long as
    // some tiles.  Measured with 3 / 4 / 5 / 6 / 7 / 8: 16 sequences up to 4091, 5 rows of 4 heads 22.1 / 21.4 / 20.9 /
    // 20.9 / 21.1 / 21.2 us, 64 up to 2048, one row 34.9 / 34.1 / 33.8 / 34.2 / 34.9 / 35.3; at 64 rows, where nearly all
    // of a segment's own work grows with them, 32 sequences up to 4096, 9 rows of 7 heads 34.2 / 33.0 / 32.4 / 32.0 / 30.8 /
    // 31.0.  Where a CTA has fewer than twice as many, half of them: few tiles are better spread.
    constexpr int kLead = N == 64 ? 7 : 5;
    // Whole parts: if there is a CTA for each task, every task may be cut into parts of its own, so that no CTA has the
    // end of one task and the beginning of another.  The parts are of `longest` tiles at most, the least that the CTAs
    // are enough for, from two up (four parts of a task, then parts of four tiles: a part more is another result to
    // join).  It is done where `longest` is no more than the equal share below would be with a segment's beginning
    // counted.  With whole parts / with equal shares, us: 16 sequences of 1000, one row 9.9 / 13.6, of 125 to 1000 10.2 /
    // 13.7; 8 of 250 to 2000, 5 rows of 4 heads 12.1 / 13.9, 9 rows of 7 15.0 / 24.3; one of 1000, one row 8.3 / 9.6.  Up
    // to 32 sequences, whose lengths the lanes keep: keeping more cost every call 0.6 us.
    // (quotients in fp32 where any near value would do; those that cut a task are whole numbers' own)
    auto over = [](int n, int d) { return (int)__fdividef((float)n + 0.25f, (float)d); };
    int longest = 0;                             // 0: equal shares
    if (each > 0 && each <= (int)gridDim.x && a.B <= 32) {
        const int most = __reduce_max_sync(0xffffffffu, mine), room = over(gridDim.x, tasks);
        auto need = [&](int t) { return (int)__reduce_add_sync(0xffffffffu, over(mine + t - 1, t)); };
        const int up = max(4, (most + 3) / 4), least = most <= 3 ? most : max(2, over(most + up - 1, up));
        int hi = max(least, over(total + each * kLead, gridDim.x)), lo = least - 1;
        if (need(hi) <= room) {
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (need(mid) <= room)
                    hi = mid;
                else
                    lo = mid;
            }
            longest = hi;
        }
    }
    const int mine_parts = longest > 0 ? (int)((uint32_t)(mine + longest - 1) / (uint32_t)longest) : 0, parts_upto = scan(mine_parts);
    if (__shfl_sync(0xffffffffu, parts_upto, 31) * tasks > (int)gridDim.x) longest = 0;     // (a quotient one off, of millions)
    int b = 0, task = 0, tile = 0;               // of the share's first tile
    int prefix = 0, before = 0;                  // tiles, and tasks, before sequence b
    int at = 0, end = 0;                         // tiles: counted from the first task's first (equal shares) or from the share's
    int parts = 0, first_cta = 0;                // of this CTA's task (whole parts)
    // Equal shares: borders i total_v / nc, rounded down (i times the remainder is below 160 x 160, and its quotient
    // by nc at least 1 / 320 from an integer after the half: fp32 finds it).  A border among a task's leading empty
    // tiles is its first tile.
    const int nc = min((int)gridDim.x, total);
    const int lead = (int)min((uint32_t)kLead, (uint32_t)total / (2u * gridDim.x));
    const int total_v = total + each * lead;
    const int share = (int)((uint32_t)total_v / (uint32_t)max(nc, 1)), rest = total_v - share * nc;
    const float per_nc = __fdividef(1.0f, (float)max(nc, 1));
    auto border_v = [&](int i) { return i * share + (int)(((float)(i * rest) + 0.5f) * per_nc); };
    auto border = [&](int v, int &sb, int &sprefix, int &sbefore, int &stask, int &stile) -> int {
        sprefix = sbefore = 0;
        for (int b0 = 0; b0 < a.B; b0 += 32) {
            const int c = b0 == 0 ? mine : b0 + lane < a.B ? tiles_of(b0 + lane) : 0, upto = b0 == 0 ? mine_upto : scan(c);
            const uint32_t there = __ballot_sync(0xffffffffu, c > 0);
            const int v_end = sprefix + sbefore * lead + (upto + __popc(there & ((2u << lane) - 1)) * lead) * tasks;
            const uint32_t past = __ballot_sync(0xffffffffu, v_end > v);
            if (past) {
                const int who = __ffs(past) - 1, cw = __shfl_sync(0xffffffffu, c, who);
                sb = b0 + who;
                sprefix += (__shfl_sync(0xffffffffu, upto, who) - cw) * tasks;
                sbefore += __popc(there & ((1u << who) - 1)) * tasks;
                const uint32_t in = (uint32_t)(v - sprefix - sbefore * lead);
                stask = (int)(in / (uint32_t)(cw + lead));
                stile = max(0, (int)in - stask * (cw + lead) - lead);
                return sprefix + stask * cw + stile;
            }
            sprefix += __shfl_sync(0xffffffffu, upto, 31) * tasks;
            sbefore += __popc(there) * tasks;
        }
        return total;
    };
    if (longest > 0) {
        const uint32_t past = __ballot_sync(0xffffffffu, parts_upto * tasks > (int)blockIdx.x);
        if (past) {
            b = __ffs(past) - 1;
            parts = __shfl_sync(0xffffffffu, mine_parts, b);
            const int first = (__shfl_sync(0xffffffffu, parts_upto, b) - parts) * tasks, tiles = __shfl_sync(0xffffffffu, mine, b);
            task = (int)((uint32_t)(blockIdx.x - first) / (uint32_t)parts);
            first_cta = first + task * parts;
            const int part = (int)blockIdx.x - first_cta;
            tile = (int)((uint32_t)(part * tiles) / (uint32_t)parts);
            end = (int)((uint32_t)((part + 1) * tiles) / (uint32_t)parts) - tile;
        }
    } else if ((int)blockIdx.x < nc) {
        end = border(border_v(blockIdx.x + 1), b, prefix, before, task, tile);
        at = border(border_v(blockIdx.x), b, prefix, before, task, tile);
    }
    int len = len_of(b), nt_task = max(1, tiles_in(len));        // the sequence's length, its tasks' tiles
    auto next = [&](int n_t) {                   // on to the next task
        at += n_t;
        tile = 0;
        if (++task == tasks && at < end) {
            task = 0;
            prefix += nt_task * tasks;
            before += tasks;
            do nt_task = tiles_in(len = len_of(++b));
            while (nt_task == 0);
        }
    };

    int loads = 0;                               // tiles whose copies were issued
    bool issued = false, elected = false;
    if (warp >= kWorkWarps) {
      asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Cfg<N>::kRegsRest));
      if (warp == kLoadWarp) {
        bool ok = true;
        while (at < end) {
            const int n_t = min(nt_task - tile, end - at), h = task / a.blocks;
            for (int i = 0; i < n_t && ok; ++i) {
                const int s = loads % kStages;
                // (after a timeout the groups free stages that they did not wait for: a copy more would meet a barrier
                // that still counts the last one; who frees a stage so has set the flag before)
                if (!(ok = all(loads < kStages ||
                               (wait(&sm.empty[s], loads / kStages + 1) && !*reinterpret_cast<volatile int *>(&sm.timeout)))))
                    break;
                if (lane == 0) {
                    umma::mbar_arrive_expect_tx(&sm.full[s], 2 * kSide);
                    umma::tma_load_3d(codes + s * 2 * kSide, &tk, 0, (tile + i) * kTok, b * a.H + h, &sm.full[s]);
                    umma::tma_load_3d(codes + s * 2 * kSide + kSide, &tv, 0, (tile + i) * kTok, b * a.H + h, &sm.full[s]);
                }
                __syncwarp();
                ++loads;
            }
            next(n_t);
        }
      } else if (warp == kTellWarp) {
        // ---- parts of tasks that others have parts of, told once their results are stored (the fence and the
        // answer would hold up the next segment for 1.4 us); told last: this CTA joins them when its tiles are done ----
        while (at < end) {
            const int n_t = min(nt_task - tile, end - at), begins = tile == 0;
            if (n_t < nt_task) {
                const int ts = prefix + task * nt_task + (before + task + 1) * lead;
                auto holder = [&](int v) {                         // the CTA whose share has place v
                    int i = (int)(__fdividef((float)nc, (float)total_v) * (float)(v + 1));     // within one
                    while (border_v(i) > v) --i;
                    while (border_v(i + 1) <= v) ++i;
                    return i;
                };
                const int c0 = longest > 0 ? first_cta : holder(ts);
                Join j{longest > 0 ? parts : holder(ts + nt_task - 1) - c0 + 1, c0, min(N, a.R * a.G - (task % a.blocks) * N), b, task};
                wait(&sm.stored[begins], 0);
                if (lane == 0) {
                    __threadfence();
                    if (atomicAdd(a.count + c0, 1) == j.parts - 1)
                        a.count[c0] = 0;                           // ready for the next call
                    else
                        j.parts = 0;
                    __threadfence();
                    sm.join[begins] = j;
                }
                __syncwarp();
            }
            next(n_t);
        }
        bar_sync(2, kWork + 32);
      } else if (warp == kScoreWarp) {
        // (the whole warp walks the loop and one lane issues: the descriptors stay in uniform registers)
        elected = umma::elect_one();
        constexpr uint32_t id = umma::instr_desc(0, 0, kTok, N);                            // f16, f32 sums
        const uint64_t qd = umma::smem_desc(umma::smem_addr(sq), N * 16, 128);
        int g = 0;
        bool ok = !stall || all(wait(&sm.drain[0], 0));             // (tests: nothing arrives there before the end)
        for (int seg = 0; at < end; ++seg) {
            const int n_t = min(nt_task - tile, end - at);
            ok = all(ok && wait(&sm.qfull, seg));
            for (int i = 0; i < n_t && ok; ++i, ++g) {
                const int s = g % kGroups;
                ok = all(wait(&sm.kfull[s], g / kGroups));
                if (!ok) break;
                umma::fence_after_sync();
                if (elected) {
#pragma unroll
                    for (int kk = 0; kk < kSteps + 1; ++kk)
                        umma::mma_bf16_ta(tmem + cS + s * N, tmem + cK + s * 80 + kk * 8, qd + (uint64_t)(kk * 2 * N), id, kk != 0);
                    umma::mma_commit(&sm.sfull[s]);
                }
                __syncwarp();
                issued = true;
            }
            next(n_t);
        }
      } else if (warp == kValueWarp) {
        elected = umma::elect_one();
        constexpr uint32_t id = umma::instr_desc(1, 1, kTok, N) | (1u << 15) | (1u << 16);  // bf16, both MN-major
        int g = 0;
        bool ok = true;
        while (at < end) {
            const int n_t = min(nt_task - tile, end - at);
            for (int i = 0; i < n_t && ok; ++i, ++g) {
                const int s = g % kGroups;
                ok = all(wait(&sm.vfull[s], g / kGroups) && wait(&sm.pfull[s], g / kGroups));
                if (!ok) break;
                umma::fence_after_sync();
                const uint64_t vd = umma::smem_desc(umma::smem_addr(sv + s * kVBuf), 128, kTok * 16);
                const uint64_t pd = umma::smem_desc(umma::smem_addr(sp + s * kP), 128, kTok * 16);
                if (elected) {
#pragma unroll
                    for (int kk = 0; kk < kTok / 16; ++kk)
                        umma::mma_bf16(tmem + cO, vd + kk * 16, pd + kk * 16, id, (i | kk) != 0);
                    umma::mma_commit(&sm.pdone[s]);
                }
                __syncwarp();
                issued = true;
            }
            if (ok && elected) umma::mma_commit(&sm.odone);
            __syncwarp();
            next(n_t);
        }
      }
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Cfg<N>::kRegsWork));
        const int grp = warp >> 2, tok = tid & (kTok - 1);
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        const uint32_t tK = tmem + lanes + cK + grp * 80, tS = tmem + lanes + cS + grp * N;
        uint8_t *const v_dst = sv + grp * kVBuf + tok * 16, *const p_dst = sp + grp * kP + tok * 16;
        // pieces of Q of a segment: row n = item / (D / 8), eight d each
        constexpr int kItems = (N * (D / 8) + kWork - 1) / kWork;
        auto q_offset = [&](int sb, int st, int n, int ld) -> long long {      // row n of task st of sequence sb
            const int hh = a.blocks == 1 ? st : st / a.blocks, nn = (st - hh * a.blocks) * N + n, r = a.row_r(nn);
            return (long long)(sb * a.R + r) * ld + (long long)(hh * a.G + (nn - r * a.G)) * D;
        };
        uint4 qx[kItems];
        auto fetch_q = [&](int sb, int st) {
            const int left = a.R * a.G - (a.blocks == 1 ? 0 : (st % a.blocks) * N);
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int it = k * kWork + tid, n = it / (D / 8);
                qx[k] = make_uint4(0, 0, 0, 0);
                if (n < N && n < left) qx[k] = __ldg(reinterpret_cast<const uint4 *>(a.q + q_offset(sb, st, n, a.ldq) + 8 * (it % (D / 8))));
            }
        };
        if (at < end) fetch_q(b, task);
        // the z step's unused columns
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%1,%1,%1,%1,%1,%1,%1};\n" ::"r"(tK + D / 2), "r"(0u) : "memory");
        umma::tmem_st_wait();
        int g = 0;                                               // tiles of this CTA so far
        for (int seg = 0; at < end; ++seg) {
            const int n_t = min(nt_task - tile, end - at);
            const int h = a.blocks == 1 ? task : task / a.blocks, row0 = (task - h * a.blocks) * N;
            const int nq = min(N, a.R * a.G - row0);
            const int p0 = tile * kTok;
            const size_t head = ((size_t)b * a.H + h) * a.T;
            // this group's tiles: i0, i0 + kGroups, ...; the scale words one tile ahead
            const int i0 = (grp + kGroups - g % kGroups) % kGroups;
            uint32_t kn = 0, vn = 0;
            if (i0 < n_t && p0 + i0 * kTok + tok < len) {
                kn = __ldg(a.ks + head + p0 + i0 * kTok + tok);
                vn = __ldg(a.vs + head + p0 + i0 * kTok + tok);
            }
            // ---- Q, rows scaled to below 2^15, in the order of unpacked codes (a thread's pieces side by side: the
            // exchanges of one after another took 0.3 us a piece) ----
            uint32_t top[kItems];
            float sum[kItems];
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const uint32_t v[4] = {qx[k].x, qx[k].y, qx[k].z, qx[k].w};
                top[k] = 0;
#pragma unroll
                for (int e = 0; e < 4; ++e) top[k] = max(top[k], max((v[e] >> 7) & 0xFFu, (v[e] >> 23) & 0xFFu));   // exponents
            }
#pragma unroll
            for (int o = D / 16; o >= 1; o >>= 1)
#pragma unroll
                for (int k = 0; k < kItems; ++k) top[k] = max(top[k], __shfl_xor_sync(0xffffffffu, top[k], o));
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int it = k * kWork + tid, n = it / (D / 8), w = it % (D / 8);
                const uint32_t v[4] = {qx[k].x, qx[k].y, qx[k].z, qx[k].w};
                top[k] = (uint32_t)min(253, 268 - (int)min(top[k], 254u));           // exponent field of 2^(14 - exponent)
                const float f = __uint_as_float(top[k] << 23), f16 = f * 0.0625f;
                float lo[4], hi[4];
                sum[k] = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    lo[e] = __uint_as_float(v[e] << 16);
                    hi[e] = __uint_as_float(v[e] & 0xFFFF0000u);
                    sum[k] += lo[e] * f + hi[e] * f;
                }
                if (n < N)
                    *reinterpret_cast<uint4 *>(sq + (w * N + n) * 16) =
                        make_uint4(pack_half(lo[0] * f, lo[2] * f), pack_half(hi[0] * f16, hi[2] * f16),
                                   pack_half(lo[1] * f, lo[3] * f), pack_half(hi[1] * f16, hi[3] * f16));
            }
#pragma unroll
            for (int o = D / 16; o >= 1; o >>= 1)
#pragma unroll
                for (int k = 0; k < kItems; ++k) sum[k] += __shfl_xor_sync(0xffffffffu, sum[k], o);
#pragma unroll
            for (int k = 0; k < kItems; ++k) {
                const int it = k * kWork + tid, n = it / (D / 8);
                if (it % (D / 8) == 0 && n < N) {
                    // z 2^-10 against -sum 2^-14 (the codes carry 2^-24), in three parts
                    const float z0 = -sum[k] * 6.103515625e-5f;
                    const __half h0 = __float2half_rn(z0), h1 = __float2half_rn(z0 - __half2float(h0)),
                                 h2 = __float2half_rn(z0 - __half2float(h0) - __half2float(h1));
                    *reinterpret_cast<uint4 *>(sq + ((D / 8) * N + n) * 16) =
                        make_uint4((uint32_t)__half_as_ushort(h0) | ((uint32_t)__half_as_ushort(h1) << 16),
                                   (uint32_t)__half_as_ushort(h2), 0u, 0u);
                    *reinterpret_cast<uint4 *>(sq + ((D / 8 + 1) * N + n) * 16) = make_uint4(0u, 0u, 0u, 0u);
                    reinterpret_cast<float *>(sm.back)[4 * (n >> 1) + (n & 1)] =
                        __uint_as_float((254u - top[k]) << 23) * (a.scale * (1.4426950408889634f * 16777216.0f));
                    sm.seen[n] = n < nq ? len - a.R + 1 + a.row_r(row0 + n) : 0;
                    sm.orow[n] = n < nq ? q_offset(b, task, n, a.ldo) : 0;
                }
            }
            umma::fence_proxy_async();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&sm.qfull);
            bar_sync(1, kWork);
            uint64_t l2[N / 2];
#pragma unroll
            for (int n = 0; n < N / 2; ++n) l2[n] = 0;
            for (int i = i0; i < n_t; i += kGroups) {
                const int gi = g + i, c = gi / kGroups, stage = gi % kStages, t = p0 + i * kTok + tok;
                const uint32_t kw = kn, vw = vn;
                kn = vn = 0;
                if (i + kGroups < n_t && t + kGroups * kTok < len) {
                    kn = __ldg(a.ks + head + t + kGroups * kTok);
                    vn = __ldg(a.vs + head + t + kGroups * kTok);
                }
                // ---- K codes into tensor memory (S^T of the group's last tile is complete: the buffer is free) ----
                wait(&sm.full[stage], gi / kStages);
                const uint8_t *kcode = codes + stage * 2 * kSide;
                uint4 x[D / 32];
#pragma unroll
                for (int y = 0; y < D / 32; ++y) x[y] = code_piece<D>(kcode, tok, y);
#pragma unroll
                for (int y = 0; y < D / 64; ++y) {
                    uint32_t r[32];
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const uint4 &xx = x[2 * y + (k >> 2)];
                        const uint32_t w = (k & 3) == 0 ? xx.x : (k & 3) == 1 ? xx.y : (k & 3) == 2 ? xx.z : xx.w, v = w >> 8;
                        r[4 * k] = w & 0x000F000Fu;
                        r[4 * k + 1] = w & 0x00F000F0u;
                        r[4 * k + 2] = v & 0x000F000Fu;
                        r[4 * k + 3] = v & 0x00F000F0u;
                    }
                    umma::tmem_st32(tK + 32 * y, r);
                }
                {
                    const uint32_t z = __half_as_ushort(__float2half_rn(hi_half(kw) * 0.0009765625f));
                    asm volatile("tcgen05.st.sync.aligned.32x32b.x2.b32 [%0], {%1,%2};\n" ::"r"(tK + D / 2), "r"(z | (z << 16)), "r"(z)
                                 : "memory");
                }
                umma::tmem_st_wait();
                umma::fence_before_sync();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&sm.kfull[grp]);
                // ---- V into its operand layout, once the products have read what was there ----
                // The bits of a code at the bottom of a bf16 lane are c 2^-133 (a subnormal), one nibble higher
                // 16 c 2^-133; one fused step brings them up by 2^127 and takes z off exactly: (c - z) 2^-6 and
                // (c - z) 2^-2.  z = 0 .. 15 whatever the word holds (fp16 z + 1024 has the integer in its low
                // bits): a bad word at an unseen place does not reach other rows as 0 times NaN.
                const float z = (float)((uint32_t)__half_as_ushort(__hadd(__ushort_as_half((uint16_t)(vw >> 16)), __ushort_as_half(0x6400))) & 15u);
                const __nv_bfloat162 up2 = __float2bfloat162_rn(1.7014118346046923e38f), z_lo = __float2bfloat162_rn(z * -0.015625f),
                                     z_hi = __float2bfloat162_rn(z * -0.25f);
#pragma unroll
                for (int y = 0; y < D / 32; ++y) x[y] = code_piece<D>(kcode + kSide, tok, y);
                // the next copy into the stage comes by the async proxy: these reads are fenced against it
                umma::fence_proxy_async();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&sm.empty[stage]);
                if (c > 0) wait(&sm.pdone[grp], c - 1);
#pragma unroll
                for (int y = 0; y < D / 32; ++y) {
                    const uint32_t ww[4] = {x[y].x, x[y].y, x[y].z, x[y].w};
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const uint32_t cc[4] = {ww[k] & 0x000F000Fu, ww[k] & 0x00F000F0u, (ww[k] >> 8) & 0x000F000Fu, (ww[k] >> 8) & 0x00F000F0u};
                        uint32_t r[4];
#pragma unroll
                        for (int f = 0; f < 4; ++f) {
                            const __nv_bfloat162 v = __hfma2(*reinterpret_cast<const __nv_bfloat162 *>(&cc[f]), up2, f & 1 ? z_hi : z_lo);
                            r[f] = *reinterpret_cast<const uint32_t *>(&v);
                        }
                        *reinterpret_cast<uint4 *>(v_dst + (4 * y + k) * (kTok * 16)) = make_uint4(r[0], r[1], r[2], r[3]);
                    }
                }
                umma::fence_proxy_async();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&sm.vfull[grp]);
                // ---- scores, p, P^T ----
                const float sk = lo_half(kw), svv = lo_half(vw);
                wait(&sm.sfull[grp], c);
                umma::fence_after_sync();
                if (i == 0 && (warp & 3) == 0) {                  // the first position's lane sets the reference
#pragma unroll
                    for (int n0 = 0; n0 < N; n0 += 16) {
                        uint32_t u[16];
                        umma::tmem_ld16(tS + n0, u);
                        umma::tmem_ld_wait();
                        if (lane == 0)
#pragma unroll
                            for (int k = 0; k < 16; k += 2)
                                reinterpret_cast<float2 *>(sm.back)[n0 + k + 1] = make_float2(-sk * __uint_as_float(u[k]), -sk * __uint_as_float(u[k + 1]));
                    }
                    if (lane == 0) umma::mbar_arrive(&sm.ref);
                }
                if (i < kGroups) wait(&sm.ref, seg);
                const uint64_t sk2 = f2(sk, sk), sv2 = f2(svv, svv);
                auto weights = [&](auto edge_c) {
                    constexpr bool kEdge = decltype(edge_c)::value;
                    constexpr int kC = N == 32 ? 32 : 16;
#pragma unroll
                    for (int n0 = 0; n0 < N; n0 += kC) {
                        if (n0 >= nq) {                           // rows past nq hold nothing
#pragma unroll
                            for (int k8 = 0; k8 < kC; k8 += 8)
                                *reinterpret_cast<uint4 *>(p_dst + ((n0 + k8) / 8) * (kTok * 16)) = make_uint4(0u, 0u, 0u, 0u);
                            continue;
                        }
                        uint32_t u[kC];
                        if constexpr (kC == 16)
                            umma::tmem_ld16(tS + n0, u);
                        else
                            umma::tmem_ld32(tS + n0, u);
                        umma::tmem_ld_wait();
#pragma unroll
                        for (int k8 = 0; k8 < kC; k8 += 8) {
                            uint32_t w[4] = {0u, 0u, 0u, 0u};
                            if (n0 + k8 < nq) {                   // (eight rows at a time)
#pragma unroll
                                for (int k = 0; k < 8; k += 2) {
                                    const int n = n0 + k8 + k;
                                    const ulonglong2 br = *reinterpret_cast<const ulonglong2 *>(&sm.back[n / 2]);
                                    const uint64_t d = mul2(br.x, fma2(sk2, f2(__uint_as_float(u[k8 + k]), __uint_as_float(u[k8 + k + 1])), br.y));
                                    float d0 = lo32(d), d1 = hi32(d);
                                    if (kEdge) {
                                        if (t >= sm.seen[n]) d0 = -INFINITY;
                                        if (t >= sm.seen[n + 1]) d1 = -INFINITY;
                                    }
                                    const float p0v = ex2(d0), p1v = ex2(d1);
                                    const uint64_t pp = f2(p0v, p1v), ws = mul2(pp, sv2);
                                    l2[n / 2] = add2(l2[n / 2], pp);
                                    // an unseen place's scale may be anything
                                    w[k / 2] = pack_bf16(kEdge && p0v == 0.0f ? 0.0f : lo32(ws), kEdge && p1v == 0.0f ? 0.0f : hi32(ws));
                                }
                            }
                            *reinterpret_cast<uint4 *>(p_dst + ((n0 + k8) / 8) * (kTok * 16)) = make_uint4(w[0], w[1], w[2], w[3]);
                        }
                    }
                };
                if (p0 + (i + 1) * kTok > len - a.R + 1)          // some row does not see some of it
                    weights(std::true_type{});
                else
                    weights(std::false_type{});
                umma::fence_before_sync();
                umma::fence_proxy_async();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&sm.pfull[grp]);
            }
            g += n_t;
            const bool whole = n_t == nt_task;
            const int seg_b = b, seg_task = task, seg_len = len;
            next(n_t);
            if (at < end) fetch_q(b, task);                       // the next segment's Q, under this one's end
            // ---- sums of p ----
            {
                float l[N];
                bool over = false;
#pragma unroll
                for (int n = 0; n < N / 2; ++n) {
                    l[2 * n] = lo32(l2[n]);
                    l[2 * n + 1] = hi32(l2[n]);
                    over |= l[2 * n] > kOver || l[2 * n + 1] > kOver;
                }
                if (over) sm.over = 1;
                lane_sums<N>(l, lane);
                if constexpr (N >= 32) {
#pragma unroll
                    for (int e = 0; e < N / 32; ++e) sm.lsum[warp][lane * (N / 32) + e] = l[e];
                } else {
                    if ((lane & 1) == 0) sm.lsum[warp][lane >> 1] = l[0];
                }
            }
            bar_sync(1, kWork);
            if (tid < N) {
                float sum = 0.0f;
#pragma unroll
                for (int w = 0; w < kWorkWarps; ++w) sum += sm.lsum[w][tid];
                const float back = reinterpret_cast<const float *>(sm.back)[4 * (tid >> 1) + (tid & 1)],
                            ref = -reinterpret_cast<const float *>(sm.back)[4 * (tid >> 1) + 2 + (tid & 1)];
                sm.inv[tid] = sum == 0.0f ? 0.0f : 1.0f / sum;                 // (NaN stays)
                sm.lse[tid] = sum == 0.0f ? kNone : fmaf(back, ref, log2f(sum));
            }
            wait(&sm.odone, seg);
            umma::fence_after_sync();
            bar_sync(1, kWork);
            // ---- results: to the output, or to this CTA's slot where others have parts of the task ----
            constexpr int kSlot = N * (D + 1);
            float *slot = a.part + ((size_t)blockIdx.x * 2 + (p0 == 0 ? 1 : 0)) * kSlot;   // (1: the task begins here)
            if (sm.over) {
                for (int n = warp; n < nq; n += kWorkWarps) {
                    float o[D / 32];
                    const float lse = plain_row<D>(a, a.q + q_offset(seg_b, seg_task, n, a.ldq), head, p0,
                                                   min(sm.seen[n], min(seg_len, p0 + n_t * kTok)), o);
#pragma unroll
                    for (int e = 0; e < D / 32; ++e) {
                        if (whole)
                            a.o[sm.orow[n] + lane * (D / 32) + e] = float_to_bf16_bits(o[e]);
                        else
                            __stcg(slot + n * D + lane * (D / 32) + e, o[e]);
                    }
                    if (!whole && lane == 0) __stcg(slot + N * D + n, lse);
                }
            } else if (32 * (warp & 3) < D) {                      // thread = d; each group every third eight rows
                const int L = 32 * (warp & 3) + lane, d = (L & ~7) | place_d(L & 7);
                const float scale = L & 2 ? 4.0f : 64.0f;          // (the operand's 2^-2 and 2^-6)
                for (int n0 = 8 * grp; n0 < nq; n0 += 8 * kGroups) {
                    uint32_t u[8];
                    umma::tmem_ld_cols<8>(tmem + lanes + cO + n0, u);
                    float inv[8];                                  // (0 where a row sees nothing; its sums are 0)
#pragma unroll
                    for (int k = 0; k < 8; k += 4) *reinterpret_cast<float4 *>(inv + k) = *reinterpret_cast<const float4 *>(sm.inv + n0 + k);
                    umma::tmem_ld_wait();
#pragma unroll
                    for (int k = 0; k < 8; ++k) inv[k] = __uint_as_float(u[k]) * (inv[k] * scale);
                    if (whole) {
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (n0 + k < nq) a.o[sm.orow[n0 + k] + d] = float_to_bf16_bits(inv[k]);
                    } else {
                        float *to = slot + n0 * D + d;
#pragma unroll
                        for (int k = 0; k < 8; ++k)
                            if (n0 + k < nq) __stcg(to + k * D, inv[k]);
                    }
                }
                umma::fence_before_sync();
                if (!whole && warp == 0)
                    for (int n = lane; n < nq; n += 32) __stcg(slot + N * D + n, sm.lse[n]);
            }
            __syncwarp();
            if (!whole && lane == 0) umma::mbar_arrive(&sm.stored[p0 == 0]);
            bar_sync(1, kWork);
            if (tid == 0) sm.over = 0;
        }
        // ---- tasks of which this CTA was the last to finish a part ----
        bar_sync(2, kWork + 32);
#pragma unroll 1
        for (int e = 0; e < 2; ++e) {
            const Join j = sm.join[e];
            if (j.parts == 0) continue;
            constexpr int kSlot = N * (D + 1), kFew = 8;
            float *wgt = reinterpret_cast<float *>(sv);             // [part][N], in the V operands' place
            auto part = [&](int c) { return a.part + ((size_t)(j.c0 + c) * 2 + (c == 0 ? 1 : 0)) * kSlot; };
            constexpr int kEach = (N * (D / 4) + kWork - 1) / kWork, kBatch = kEach < 3 ? 4 : 2;   // loads in flight: kEach x kBatch
            float4 x[kEach], y[kBatch][kEach];
            auto fetch = [&](int cb) {
#pragma unroll
                for (int c = 0; c < kBatch; ++c)
#pragma unroll
                    for (int k = 0; k < kEach; ++k) {
                        const int it = k * kWork + tid;
                        y[c][k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
                        if (cb + c < j.parts && it < j.nq * (D / 4)) y[c][k] = __ldcg(reinterpret_cast<const float4 *>(part(cb + c)) + it);
                    }
            };
            fetch(0);                                               // (under the weights)
            if (j.parts <= kFew) {                                  // a thread per row
                if (tid < j.nq) {
                    float v[kFew], top = kNone, sum = 0.0f;
#pragma unroll
                    for (int c = 0; c < kFew; ++c) v[c] = c < j.parts ? __ldcg(part(c) + N * D + tid) : kNone;
#pragma unroll
                    for (int c = 0; c < kFew; ++c) top = fmaxf(top, v[c]);
#pragma unroll
                    for (int c = 0; c < kFew; ++c) {
                        v[c] = v[c] == kNone ? 0.0f : ex2(v[c] - top);          // (NaN stays)
                        sum += v[c];
                    }
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                    for (int c = 0; c < kFew; ++c)
                        if (c < j.parts) wgt[c * N + tid] = v[c] * inv;
                }
            } else {                                                // a warp per row
                for (int n = warp; n < j.nq; n += kWorkWarps) {
                    float v[(kMaxCtas + 31) / 32], top = kNone, sum = 0.0f;
#pragma unroll
                    for (int k = 0; k < (kMaxCtas + 31) / 32; ++k) {
                        v[k] = 32 * k + lane < j.parts ? __ldcg(part(32 * k + lane) + N * D + n) : kNone;
                        top = fmaxf(top, v[k]);
                    }
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
#pragma unroll
                    for (int k = 0; k < (kMaxCtas + 31) / 32; ++k) {
                        v[k] = v[k] == kNone ? 0.0f : ex2(v[k] - top);
                        sum += v[k];
                    }
#pragma unroll
                    for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                    const float inv = sum == 0.0f ? 0.0f : 1.0f / sum;
#pragma unroll
                    for (int k = 0; k < (kMaxCtas + 31) / 32; ++k)
                        if (32 * k + lane < j.parts) wgt[(32 * k + lane) * N + n] = v[k] * inv;
                }
            }
            bar_sync(1, kWork);
#pragma unroll
            for (int k = 0; k < kEach; ++k) x[k] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
            for (int cb = 0; cb < j.parts; cb += kBatch) {
                if (cb > 0) fetch(cb);
#pragma unroll
                for (int c = 0; c < kBatch; ++c)
#pragma unroll
                    for (int k = 0; k < kEach; ++k) {
                        const int it = k * kWork + tid;
                        if (cb + c < j.parts && it < j.nq * (D / 4)) {
                            const float w = wgt[(cb + c) * N + it / (D / 4)];
                            x[k].x = fmaf(w, y[c][k].x, x[k].x), x[k].y = fmaf(w, y[c][k].y, x[k].y);
                            x[k].z = fmaf(w, y[c][k].z, x[k].z), x[k].w = fmaf(w, y[c][k].w, x[k].w);
                        }
                    }
            }
#pragma unroll
            for (int k = 0; k < kEach; ++k) {
                const int it = k * kWork + tid, n = it / (D / 4);
                if (n < j.nq)
                    *reinterpret_cast<uint2 *>(a.o + q_offset(j.b, j.task, n, a.ldo) + 4 * (it % (D / 4))) =
                        make_uint2(pack_bf16(x[k].x, x[k].y), pack_bf16(x[k].z, x[k].w));
            }
            bar_sync(1, kWork);
        }
    }

    // after a timeout: copies and products in flight finish (bounded) before
    // the memory is released
    __syncthreads();
    if (sm.timeout) {
        if (warp == kLoadWarp && lane == 0)
            for (int i = max(0, loads - kStages); i < loads; ++i)
                umma::mbar_wait(&sm.full[i % kStages], (uint32_t)((i / kStages) & 1), kWaitLimit);
        if ((warp == kScoreWarp || warp == kValueWarp) && elected && issued) {
            umma::mma_commit(&sm.drain[warp - kScoreWarp]);
            umma::mbar_wait(&sm.drain[warp - kScoreWarp], 0, kWaitLimit);
        }
        if (tid == 0) flag(a.st, QSPEC_ERR_TIMEOUT);
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == kScoreWarp) umma::tmem_free(tmem, kCols);
}

bool sizes_ok(int B, int R, int Hq, int H, int D) {
    return B >= 1 && R >= 1 && R <= kMaxR && H >= 1 && Hq >= H && Hq % H == 0 && (D == 64 || D == 128) &&
           Hq / H <= 8192 && (long long)B * R * Hq < (1LL << 28);
}

constexpr size_t kCountBytes = kMaxCtas * sizeof(int);
constexpr size_t kPartBytes = (size_t)kMaxCtas * 2 * kMaxN * (kMaxD + 1) * sizeof(float);

template <int D, int N>
int launch(Args a, cudaStream_t stream, uint32_t wait_limit, int stall) {
    a.blocks = (a.R * a.G + N - 1) / N;
    CUtensorMap tk, tv;
    if (code_tmap(&tk, a.kc, D / 2, a.T, a.B * a.H, kTok) || code_tmap(&tv, a.vc, D / 2, a.T, a.B * a.H, kTok))
        return QSPEC_ERR_UNSUPPORTED;
    auto kern = attn_kv4_kernel<D, N>;
    int rc = smem_limit_once(reinterpret_cast<const void *>(kern), (int)smem_bytes<D, N>());
    if (rc) return rc;
    const long long most = (long long)a.B * a.H * a.blocks * std::max(1, (a.T + kTok - 1) / kTok);   // tiles at full lengths
    const unsigned grid = (unsigned)std::min<long long>(std::min(sm_count(), kMaxCtas), most);
    return launch_pdl("qspec_attn_kv4", kern, dim3(grid), dim3(Cfg<N>::kThreads), smem_bytes<D, N>(), stream, tk, tv, a,
                      wait_limit, stall);
}

// rows per pass: the fewest passes over the cache, then the narrowest that holds them
template <int D>
int dispatch(const Args &a, cudaStream_t stream, uint32_t wait_limit, int stall) {
    const int rows = a.R * a.G, passes = (rows + kMaxN - 1) / kMaxN, each = (rows + passes - 1) / passes;
    if (each <= 16) return launch<D, 16>(a, stream, wait_limit, stall);
    if (each <= 32) return launch<D, 32>(a, stream, wait_limit, stall);
    return launch<D, 64>(a, stream, wait_limit, stall);
}

}  // namespace akv

}  // namespace

}  // namespace qspec

using namespace qspec;

extern "C" size_t qspec_attn_kv4_workspace_bytes(int B, int R, int Hq, int H, int D) {
    // the same for every shape: arrival counts, then two partial results per CTA
    return akv::sizes_ok(B, R, Hq, H, D) ? akv::kCountBytes + akv::kPartBytes : 0;
}

extern "C" int qspec_debug_attn_kv4_bounded(const uint16_t *q_bf16, int ldq, const uint8_t *k_codes, const uint32_t *k_sz,
                                            const uint8_t *v_codes, const uint32_t *v_sz, const int32_t *len, int B, int R,
                                            int Hq, int H, int T, int D, float scale, uint16_t *o_bf16, int ldo,
                                            void *workspace, size_t ws_bytes, uint32_t wait_limit, int stall,
                                            int32_t *dev_status, qspec_stream_t stream) {
    if (!q_bf16 || !k_codes || !k_sz || !v_codes || !v_sz || !len || !o_bf16 || !workspace) return QSPEC_ERR_NULL;
    if (!akv::sizes_ok(B, R, Hq, H, D) || T < 1 || T > (1 << 30) || (long long)B * H >= (1LL << 31) ||
        !std::isfinite(scale) || ldq < (long long)Hq * D || ldo < (long long)Hq * D || wait_limit < 1)
        return QSPEC_ERR_SHAPE;
    // tiles of all tasks, the empty ones in front of each counted, are 32-bit numbers in the kernel
    const long long passes = (R * (long long)(Hq / H) + akv::kMaxN - 1) / akv::kMaxN;
    if (B * (long long)H * passes * ((T + akv::kTok - 1) / akv::kTok + 8) >= (1LL << 30)) return QSPEC_ERR_SHAPE;
    if (ldq % 8 || ldo % 8 || !aligned(q_bf16, 16) || !aligned(o_bf16, 16) || !aligned(k_codes, 16) ||
        !aligned(v_codes, 16) || !aligned(k_sz, 4) || !aligned(v_sz, 4) || !aligned(len, 4) || !aligned(workspace, 16))
        return QSPEC_ERR_ALIGN;
    if (ws_bytes < qspec_attn_kv4_workspace_bytes(B, R, Hq, H, D)) return QSPEC_ERR_WORKSPACE;
    int rc = check_device();
    if (rc) return rc;
    const akv::Args a{q_bf16, k_codes, v_codes, k_sz, v_sz, len, o_bf16, dev_status, reinterpret_cast<int *>(workspace),
                      reinterpret_cast<float *>(static_cast<uint8_t *>(workspace) + akv::kCountBytes), ldq, ldo, B, R,
                      Hq / H, H, T, 1, Hq == H ? 0u : (uint32_t)((1ull << 32) / (Hq / H) + 1), scale};
    return D == 128 ? akv::dispatch<128>(a, as_cuda(stream), wait_limit, stall)
                    : akv::dispatch<64>(a, as_cuda(stream), wait_limit, stall);
}

extern "C" int qspec_attn_kv4(const uint16_t *q_bf16, int ldq, const uint8_t *k_codes, const uint32_t *k_sz,
                              const uint8_t *v_codes, const uint32_t *v_sz, const int32_t *len, int B, int R, int Hq,
                              int H, int T, int D, float scale, uint16_t *o_bf16, int ldo, void *workspace,
                              size_t ws_bytes, int32_t *dev_status, qspec_stream_t stream) {
    return qspec_debug_attn_kv4_bounded(q_bf16, ldq, k_codes, k_sz, v_codes, v_sz, len, B, R, Hq, H, T, D, scale, o_bf16,
                                        ldo, workspace, ws_bytes, kWaitLimit, 0, dev_status, stream);
}
