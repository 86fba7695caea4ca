// attn_prompt.cu -- causal attention of packed prompts, grouped heads, on the
// Blackwell tensor cores.
//
//   a_ij = scale q_i . k_j for j <= i + Lk - Lq,  o_i = sum_j softmax(a_i)_j v_j
//
// The Lq G query rows that read one KV head (row-major position, head of the
// group minor) form one matrix, cut into tiles of 128 rows whatever G is; a CTA
// takes two consecutive tiles, so each key tile of 128 rows is read once for 256
// rows and both tiles end at nearly the same key.  Per key tile and row tile t:
//   S_t = Q_t K^T (tcgen05, both operands in shared memory, S in tensor memory),
//   the softmax warps of t read S_t (thread = row) and write p = 2^(c s - m) as
//   bf16 over S_t in tensor memory, in two halves, and keep the sum l,
//   O_t += P_t V (P from tensor memory, V rows as they are: an MN-major operand).  P is
//   bf16 because V is (a product takes one type); its sum l is of the fp32 weights.
// The issuing lane interleaves the two tiles, so one tile's softmax runs under
// the other's products.
// The reference m is the row's maximum over the first key tile and after that follows
// the sums instead of the maxima: where a tile's sum of p passes 2^12, the next tile
// begins by moving m up (by a power of two, exactly) and rescaling l and O_t.  No
// pass over the scores looks for their maximum, and nothing is lost meanwhile, p and O
// being floating point; a score that passes m by some 2^90 within one tile ends
// in a result that is not finite, and such rows are computed again.  The softmax
// warps rescale O_t themselves: the completed product S_t(i + 1) implies that
// O_t += P_t(i) V has completed, so no other synchronisation is needed for it.
//
// CTAs are persistent: one warp finds a CTA's units (the longest first) and fetches
// their queries ahead, so the next unit's copies run under the present one's products.
//
// Bound: tensor cores and shared memory at once (D = 128): a pair of row tiles and a
// key tile are 2093 clocks of products (measured: 62 to 68 for N = 128) and 256 KB of
// shared memory (128 of them Q and K for the scores, 64 V, 64 the copies' writes), 2048
// clocks at 128 bytes each; together they take some 2650.  What adds shared-memory
// operations costs more than it hides (8192 tokens, 342 us as it is): waits
// that spin 398, weights handed over in three parts 374, two warpgroups to a row
// tile 408; with the exponentials left out it was as long.  8192 tokens, 8 KV heads
// of 128 with 4 heads each: 365 to 373 us a call with new inputs, 342 to 359 in a
// captured graph (from one GPU to another), that is 1480 to 1607 TFLOP/s counting what
// the mask leaves; 7 sequences of 5003 tokens, 4 KV heads with 7 each: 50 us; 3 of 301: 7.5 us.
#include <algorithm>
#include <cmath>

#include "qspec_device.cuh"
#include "qspec_host.h"
#include "umma.cuh"

namespace qspec {

namespace {

namespace apr {

constexpr int kTile = 128;                      // query rows per tile, keys per tile
constexpr int kSoftmax = 256;                   // softmax threads: 128 per row tile
constexpr int kMmaWarp = kSoftmax / 32, kTmaWarp = kMmaWarp + 1;
constexpr int kUnitWarp = kTmaWarp + 1;         // finds the units and fetches their Q (one more warp idles: register
                                                // shares are given to four warps at a time)
constexpr int kThreads = kSoftmax + 128;
// registers per thread: 384 threads start with 168 and share 64512
constexpr int kRegsStart = 168, kRegsSoftmax = 216, kRegsRest = 64;
static_assert(kSoftmax * kRegsSoftmax + 128 * kRegsRest <= kThreads * kRegsStart, "register shares");
constexpr uint32_t kCols = 512;                 // tensor memory: S0, S1 (128 columns each), O0, O1 (D each)
constexpr uint32_t kS = 0, kO = 256;
constexpr float kGrown = 4096.0f;               // a tile's sum of p from where the reference moves

template <int D>
constexpr int tile_bytes() { return kTile * D * 2; }
template <int D>
constexpr int ring() { return D == 128 ? 4 : 8; }

struct Unit {
    int h, q0, k0, off;                         // group of heads, the sequence's first rows, Lk - Lq
    int first, left, n;                         // first position, positions from it on (to the sequence's end), key tiles; n < 0: no more units
};

struct Ctl {
    uint64_t full[8], empty[8];                 // K / V tiles: landed, read
    uint64_t ufull[2], uempty[2];               // units: published, done with
    uint64_t qfull[2], qfree[2];                // Q tiles: written, read
    uint64_t sfull[2], pfull[2][2], odone[2];   // S_t written, each half of P_t written (and S_t read), O_t complete
    uint64_t drain;
    Unit unit[2];
    uint32_t tmem;
    int timeout, q_count[2];
};

constexpr int kOutBytes = kSoftmax / 32 * 32 * 128;   // per softmax warp 32 rows x 64 values on their way out
template <int D>
constexpr size_t smem_total() { return 1024 + 2 * (size_t)tile_bytes<D>() + (size_t)ring<D>() * tile_bytes<D>() + kOutBytes + sizeof(Ctl); }

struct Args {
    const uint16_t *q, *k, *v;
    const int32_t *q_start, *k_start;
    uint16_t *o;
    int32_t *st;
    int ldq, ldk, ldv, ldo, q_rows, k_rows, B, H, G;   // H groups of G query heads
    int share;                                  // groups to a KV head
    uint32_t g_mul;                             // n / G = umulhi(n, g_mul) for n < 128 (G = 1: 0)
    float scale;

    __device__ __forceinline__ int over_g(int n) const { return g_mul ? (int)__umulhi((uint32_t)n, g_mul) : n; }
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

__device__ __forceinline__ float max3(float a, float b, float c) {
    float r;
    asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
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

// K-major operand, 128-byte swizzle: 8 rows x 128 bytes per 1024-byte atom, the
// row groups 1024 bytes apart (rows of 64 bf16; the next 64 one box further)
__device__ __forceinline__ uint64_t desc_k(uint32_t saddr) {
    return umma::smem_desc(saddr, 16, 1024) | ((uint64_t)2 << 61);
}
// MN-major operand (V as it lies: rows = K dimension), 128-byte swizzle: 64
// values of the MN dimension per 128-byte row, the next 64 one box (kTile rows)
// further, groups of 8 rows 1024 bytes apart
__device__ __forceinline__ uint64_t desc_mn(uint32_t saddr) {
    return umma::smem_desc(saddr, kTile * 128, 1024) | ((uint64_t)2 << 61);
}

// the bits 15 and 31 of two bf16 values that are not finite
__device__ __forceinline__ uint32_t not_finite(uint32_t w) { return ((w & 0x7F807F80u) + 0x00800080u) & 0x80008000u; }

// Rows of a warp (its lanes `walk`) from the keys that each sees only, four together: eight lanes to a row, which take
// every eighth 16 bytes of a key, staged eight keys at a time in the warp's 4 KB `buf`.  (Four lanes to a row are
// faster here, but with the registers they need the kernel's own loop spills: 353 us for 344 at 8192 rows.)
// `suspect`: the first key that holds something that is not finite; where some score has no softmax, nor has the row.
template <int D>
__device__ __noinline__ void rows_by_key(const Args &a, int hg, int q0, int k0, int off, int p, int g, int suspect, uint32_t walk, uint4 *buf) {
    constexpr int kLanes = 8, C = D / (8 * kLanes), P = 4 * C;          // lanes to a row; their 16-byte pieces of it, pairs of values
    constexpr int J = 8, L = J * D / 256;                               // keys at a time; a lane's loads of them
    static_assert(2 * J * D * 2 <= kOutBytes / (kSoftmax / 32), "K and V of J keys in a warp's part");
    const int lane = threadIdx.x & 31, part = lane % kLanes, h = hg / a.share;
    const uint16_t *kc = a.k + (size_t)k0 * a.ldk + (size_t)h * D, *vc = a.v + (size_t)k0 * a.ldv + (size_t)h * D;
    auto unpack = [](const uint4 &w, uint64_t *to) {
        const uint32_t v[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) to[i] = f2(__uint_as_float(v[i] << 16), __uint_as_float(v[i] & 0xFFFF0000u));
    };
    auto pairs = [&](const uint16_t *row, uint64_t (&to)[P]) {          // this lane's values of a row of D
#pragma unroll
        for (int i = 0; i < C; ++i) unpack(*reinterpret_cast<const uint4 *>(row + 8 * (kLanes * i + part)), to + 4 * i);
    };
    const float c = a.scale * 1.4426950408889634f;
    auto score = [&](uint64_t s) {                                      // in log2 units
        float v = lo32(s) + hi32(s);
#pragma unroll
        for (int x = 1; x < kLanes; x <<= 1) v += __shfl_xor_sync(0xffffffffu, v, x);
        return v * c;
    };
    while (walk) {
        int who = -1;                                                   // this row's lane in the mask, -1: none
#pragma unroll
        for (int r = 0; r < 32 / kLanes; ++r, walk &= walk - 1)
            if (r == lane / kLanes && walk) who = __ffs(walk) - 1;
        const int from = max(who, 0), pw = __shfl_sync(0xffffffffu, p, from), gw = __shfl_sync(0xffffffffu, g, from);
        const int lim = who < 0 ? -1 : pw + off, most = __reduce_max_sync(0xffffffffu, lim);
        const size_t hw = (size_t)(hg * a.G + gw) * D;
        uint64_t q[P], acc[P];
        pairs(a.q + (size_t)(q0 + pw) * a.ldq + hw, q);
        float m = -INFINITY, l = 0.0f;
        bool bad = false;
        if (suspect <= most) {
            uint64_t k[P], s = 0;
            pairs(kc + (size_t)suspect * a.ldk, k);
#pragma unroll
            for (int i = 0; i < P; ++i) s = fma2(q[i], k[i], s);
            bad = !(score(s) < INFINITY) && suspect <= lim;
        }
#pragma unroll
        for (int i = 0; i < P; ++i) acc[i] = 0;
        uint4 next[2][L];
        auto fetch = [&](int j0) {                                      // (past the last key: that again, not used)
#pragma unroll
            for (int x = 0; x < L; ++x) {
                const int it = x * 32 + lane, j = min(j0 + it / (D / 8), most), d = 8 * (it % (D / 8));
                next[0][x] = *reinterpret_cast<const uint4 *>(kc + (size_t)j * a.ldk + d);
                next[1][x] = *reinterpret_cast<const uint4 *>(vc + (size_t)j * a.ldv + d);
            }
        };
        fetch(0);
        for (int j0 = 0; j0 <= most && !__all_sync(0xffffffffu, bad || lim < j0); j0 += J) {
            __syncwarp();
#pragma unroll
            for (int side = 0; side < 2; ++side)
#pragma unroll
                for (int x = 0; x < L; ++x) buf[side * (J * D / 8) + x * 32 + lane] = next[side][x];
            __syncwarp();
            fetch(j0 + J);
            auto piece = [&](int side, int j, int i, uint64_t (&to)[4]) { unpack(buf[(side * J + j) * (D / 8) + kLanes * i + part], to); };
            float s[J], m1 = m;
#pragma unroll
            for (int j = 0; j < J; ++j) {
                uint64_t two = 0;
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    uint64_t k[4];
                    piece(0, j, i, k);
#pragma unroll
                    for (int e = 0; e < 4; ++e) two = fma2(q[4 * i + e], k[e], two);
                }
                s[j] = score(two);
                if (j0 + j > lim) s[j] = -INFINITY;
                bad |= !(s[j] < INFINITY);
                m1 = fmaxf(m1, s[j]);
            }
            const float ref = m1 > -INFINITY ? m1 : 0.0f, f = ex2(m - ref);
            m = m1;
            l *= f;
#pragma unroll
            for (int i = 0; i < P; ++i) acc[i] = mul2(acc[i], f2(f, f));
#pragma unroll
            for (int j = 0; j < J; ++j) {
                if (j0 + j > lim) continue;                             // (0 times a NaN of an unseen key)
                const float pj = ex2(s[j] - ref);
                l += pj;
#pragma unroll
                for (int i = 0; i < C; ++i) {
                    uint64_t v[4];
                    piece(1, j, i, v);
#pragma unroll
                    for (int e = 0; e < 4; ++e) acc[4 * i + e] = fma2(f2(pj, pj), v[e], acc[4 * i + e]);
                }
            }
        }
        if (who >= 0) {
            const float inv = bad ? NAN : l == 0.0f ? 0.0f : 1.0f / l;
            uint16_t *orow = a.o + (size_t)(q0 + pw) * a.ldo + hw + 8 * part;
            auto out = [&](int i) { return pack_bf16(lo32(acc[i]) * inv, hi32(acc[i]) * inv); };
#pragma unroll
            for (int i = 0; i < C; ++i)
                *reinterpret_cast<uint4 *>(orow + 8 * kLanes * i) = make_uint4(out(4 * i), out(4 * i + 1), out(4 * i + 2), out(4 * i + 3));
        }
    }
}

// The rows `again` of a warp, whose results are not finite.  Three things make them so: the row sees such a value
// and its result is right; a weight of 0 met a NaN or inf of an unseen key (a masked place of the last key
// tiles); a score passed the reference by more than fp32 holds.  The last two are computed again.  The first is
// told from them by one look at what the rows see, for all rows of the warp together: a NaN sum of weights comes
// from a score, and a value of o from a seen V that is not finite in its dimension.  With every such row computed
// again one NaN in an early row of V took 4096 rows from 0.10 ms to 100; it is 0.39, and 2.8 with a NaN half way, for
// the rows before it in its own key tile.
template <int D>
__device__ __noinline__ void rows_again(const Args &a, int hg, int q0, int k0, int off, int p, int g, float l, uint32_t again) {
    constexpr int C = D / 8, kKeys = 32 / C, kAhead = 8;                // lanes to a row, 16 bytes each; keys a load; loads
    const int lane = threadIdx.x & 31, h = hg / a.share;
    const size_t col = (size_t)h * D + 8 * (lane % C);
    const uint16_t *kc = a.k + (size_t)k0 * a.ldk + col, *vc = a.v + (size_t)k0 * a.ldv + col;
    auto at = [](const uint16_t *row) { return *reinterpret_cast<const uint4 *>(row); };
    auto marks = [](const uint4 &w) { return make_uint4(not_finite(w.x), not_finite(w.y), not_finite(w.z), not_finite(w.w)); };
    uint4 bad = make_uint4(0, 0, 0, 0);                                 // this lane's dimensions with such a value of V
    uint32_t walk = 0;
    int suspect = 0x7FFFFFFF, upto = 0;                                 // first such key of K; keys looked at
    while (again) {                                                     // (rows further on see more)
        const int who = __ffs(again) - 1;
        again &= again - 1;
        const int pw = __shfl_sync(0xffffffffu, p, who), gw = __shfl_sync(0xffffffffu, g, who), lim = pw + off;
        const float lw = __shfl_sync(0xffffffffu, l, who);
        if (lw == -1.0f) continue;                                      // (a score is NaN)
        for (; upto <= lim; upto += kKeys * kAhead) {
            uint4 kw[kAhead], vw[kAhead];
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const size_t j = min(upto + i * kKeys + lane / C, lim);
                kw[i] = at(kc + j * a.ldk);
                vw[i] = at(vc + j * a.ldv);
            }
#pragma unroll
            for (int i = 0; i < kAhead; ++i) {
                const uint4 k = marks(kw[i]), v = marks(vw[i]);
                if (k.x | k.y | k.z | k.w) suspect = min(suspect, min(upto + i * kKeys + lane / C, lim));
                bad = make_uint4(bad.x | v.x, bad.y | v.y, bad.z | v.z, bad.w | v.w);
            }
        }
        upto = lim + 1;
#pragma unroll
        for (int o = C; o < 32; o <<= 1) {
            bad.x |= __shfl_xor_sync(0xffffffffu, bad.x, o), bad.y |= __shfl_xor_sync(0xffffffffu, bad.y, o);
            bad.z |= __shfl_xor_sync(0xffffffffu, bad.z, o), bad.w |= __shfl_xor_sync(0xffffffffu, bad.w, o);
        }
        const uint4 r = marks(at(a.o + (size_t)(q0 + pw) * a.ldo + (size_t)(hg * a.G + gw) * D + 8 * (lane % C)));
        const bool other = !(lw > 0.0f && lw < INFINITY) || ((r.x & ~bad.x) | (r.y & ~bad.y) | (r.z & ~bad.z) | (r.w & ~bad.w));
        if (__any_sync(0xffffffffu, other)) walk |= 1u << who;
    }
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *so = smem_raw + ((1024u - (umma::smem_addr(smem_raw) & 1023u)) & 1023u) + (2 + ring<D>()) * tile_bytes<D>();
    if (walk)
        rows_by_key<D>(a, hg, q0, k0, off, p, g, __reduce_min_sync(0xffffffffu, suspect), walk,
                       reinterpret_cast<uint4 *>(so + (threadIdx.x >> 5) * (32 * 128)));
}

template <int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_prompt_kernel(const __grid_constant__ CUtensorMap tq, const __grid_constant__ CUtensorMap tk,
                       const __grid_constant__ CUtensorMap tv,
                       const __grid_constant__ Args a,
                       uint32_t wait_limit, int stall) {
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    constexpr int kT = tile_bytes<D>(), NS = ring<D>();
    // (an offset, not a rounded address: the compiler keeps seeing shared memory)
    uint8_t *sq = smem_raw + ((1024u - (umma::smem_addr(smem_raw) & 1023u)) & 1023u);
    uint8_t *skv = sq + 2 * kT;
    uint8_t *so = skv + NS * kT;
    Ctl &sm = *reinterpret_cast<Ctl *>(so + kOutBytes);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int G = a.G, per_tile = kTile / G;                // positions to a row tile

    if (warp == kMmaWarp) umma::tmem_alloc(&sm.tmem, kCols);
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            umma::mbar_init(&sm.full[s], 1);
            umma::mbar_init(&sm.empty[s], 1);
        }
        for (int t = 0; t < 2; ++t) {
            umma::mbar_init(&sm.sfull[t], 1);
            umma::mbar_init(&sm.pfull[t][0], kTile / 32);
            umma::mbar_init(&sm.pfull[t][1], kTile / 32);
            umma::mbar_init(&sm.odone[t], 1);
            umma::mbar_init(&sm.ufull[t], 1);
            umma::mbar_init(&sm.uempty[t], kSoftmax / 32 + 2);          // softmax, products, copies
            umma::mbar_init(&sm.qfull[t], 1);
            umma::mbar_init(&sm.qfree[t], 1);
        }
        umma::mbar_init(&sm.drain, 1);
        sm.timeout = 0;
        umma::mbar_fence_init();
    }
    pdl_launch_dependents();
    pdl_wait();
    // the first 32 sequences' rows (asked for before the barrier)
    int4 rows = make_int4(0, 0, 0, 0);
    if (warp == kUnitWarp && lane < a.B)
        rows = make_int4(__ldg(a.q_start + lane), __ldg(a.q_start + lane + 1), __ldg(a.k_start + lane), __ldg(a.k_start + lane + 1));
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    const uint32_t tmem = sm.tmem;

    int loads = 0;
    bool issued = false, elected = false;
    auto wait = [&](uint64_t *bar, uint32_t phase) -> bool {
        if (umma::mbar_try_wait(bar, phase & 1)) return true;
        if (*reinterpret_cast<volatile int *>(&sm.timeout)) return false;
        if (umma::mbar_wait(bar, phase & 1, wait_limit)) return true;
        *reinterpret_cast<volatile int *>(&sm.timeout) = 1;
        return false;
    };
    // (the votes keep a warp together where a wait runs out)
    auto all = [](bool mine) { return __all_sync(0xffffffffu, mine) != 0; };
    int span = 0;                                           // positions to a unit (of the warp that finds them)
    auto tiles = [&](const Unit &u) { return u.left > per_tile ? 2 : 1; };  // row tiles with rows

    if (warp >= kMmaWarp) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsRest));
        if (warp == kUnitWarp) {
            // ---- units: level by level from the sequences' last ones (the longest), for up to 32 sequences;
            // for more, sequence by sequence, each one's last unit first ----
            {
                int q0 = 0, lq = 0, k0 = 0, lk = 0;
                auto fetch = [&](int b, bool report) {
                    q0 = lq = k0 = lk = 0;
                    if (b >= a.B) return;
                    const int q1 = b < 32 ? rows.y : __ldg(a.q_start + b + 1), k1 = b < 32 ? rows.w : __ldg(a.k_start + b + 1);
                    q0 = b < 32 ? rows.x : __ldg(a.q_start + b);
                    k0 = b < 32 ? rows.z : __ldg(a.k_start + b);
                    if (q0 < 0 || q1 < q0 || q1 > a.q_rows || k0 < 0 || k1 < k0 || k1 > a.k_rows) {
                        if (report) flag(a.st, QSPEC_ERR_RANGE);
                        return;
                    }
                    lq = q1 - q0;
                    lk = k1 - k0;
                };
                auto units_of = [&](int positions) { return (lq + positions - 1) / positions; };
                int total[2] = {0, 0};                                  // units of one tile, of two (times H: the host keeps it
                                                                        // below 2^31)
                for (int b0 = 0; b0 < a.B; b0 += 32) {
                    fetch(b0 + lane, blockIdx.x == 0);
                    total[0] += __reduce_add_sync(0xffffffffu, units_of(per_tile));
                    total[1] += __reduce_add_sync(0xffffffffu, units_of(2 * per_tile));
                }
                if (a.B > 32) fetch(lane, false);
                const bool one = (uint32_t)(total[0] * a.H) <= gridDim.x;           // one tile each still leaves SMs idle
                span = one ? per_tile : 2 * per_tile;
                const uint32_t end = (uint32_t)((one ? total[0] : total[1]) * a.H);
                int count[2] = {0, 0};                                  // Q tiles fetched
                bool ok = true;
                for (int k = 0;; ++k) {
                    const uint32_t id = k * gridDim.x + (k & 1 ? gridDim.x - 1 - blockIdx.x : blockIdx.x);
                    const bool more = id < end;
                    if (k >= 2 && !all(wait(&sm.uempty[k & 1], (k >> 1) - 1))) break;
                    Unit &u = sm.unit[k & 1];
                    bool mine = false;
                    int index = 0;
                    const uint32_t place = id / (uint32_t)a.H;
                    if (more) {
                        int rank = (int)place;
                        if (a.B <= 32) {
                            const int units = units_of(span);
                            auto from = [&](int level) { return (int)__reduce_add_sync(0xffffffffu, max(0, units - level)); };   // units at level and above
                            int lo = 0, hi = (int)__reduce_max_sync(0xffffffffu, units);
                            while (hi - lo > 1) {
                                const int mid = (lo + hi) >> 1;
                                if (from(mid) > rank)
                                    lo = mid;
                                else
                                    hi = mid;
                            }
                            rank -= from(lo + 1);
                            const uint32_t there = __ballot_sync(0xffffffffu, units > lo);
                            mine = units > lo && __popc(there & ((1u << lane) - 1)) == rank;
                            index = lo;
                        } else {
                            for (int b0 = 0; b0 < a.B && rank >= 0; b0 += 32) {
                                fetch(b0 + lane, false);
                                const int units = units_of(span);
                                int upto = units;
#pragma unroll
                                for (int x = 1; x < 32; x <<= 1) {
                                    const int y = __shfl_up_sync(0xffffffffu, upto, x);
                                    if (lane >= x) upto += y;
                                }
                                const int sum = __shfl_sync(0xffffffffu, upto, 31);
                                mine = rank >= upto - units && rank < upto;
                                index = units - 1 - (rank - (upto - units));
                                rank = rank < sum ? -1 : rank - sum;
                            }
                        }
                    }
                    if (mine) {
                        u.h = (int)(id - place * a.H);
                        u.q0 = q0;
                        u.k0 = k0;
                        u.off = lk - lq;
                        u.first = index * span;
                        u.left = min(lq - u.first, span);
                        u.n = max(0, (u.first + u.left - 1 + u.off + kTile) / kTile);    // that its last row sees
                    }
                    if (!more && lane == 0) u.n = -1;
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(&sm.ufull[k & 1]);
                    if (!more) break;
                    // its Q tiles: whole positions' heads in one box of 64 values each (rows past the sequence hold
                    // whatever follows; their scores are all masked)
                    for (int t = 0; t < tiles(u) && u.n > 0 && ok; ++t) {
                        if (count[t] > 0 && !(ok = all(wait(&sm.qfree[t], count[t] - 1)))) break;
                        if (lane == 0) {
                            umma::mbar_arrive_expect_tx(&sm.qfull[t], per_tile * G * D * 2);
#pragma unroll
                            for (int c = 0; c < D / 64; ++c)
                                umma::tma_load_3d(sq + t * kT + c * (kTile * 128), &tq, 128 * c, u.h * G, u.q0 + u.first + t * per_tile, &sm.qfull[t]);
                        }
                        ++count[t];
                        __syncwarp();
                    }
                    if (!ok) break;
                }
                if (lane == 0)                                          // (for the drain after a timeout)
                    for (int t = 0; t < 2; ++t) sm.q_count[t] = count[t];
            }
        } else if (warp == kTmaWarp) {
            bool ok = true;
            for (int k = 0; ok; ++k) {
                if (!(ok = all(wait(&sm.ufull[k & 1], k >> 1)))) break;
                const Unit &u = sm.unit[k & 1];
                const int n = u.n, h = a.share == 1 ? u.h : u.h / a.share, k0 = u.k0;
                if (n < 0) break;
                for (int i = 0; i < 2 * n && ok; ++i, ++loads) {       // K_0, V_0, K_1, V_1, ...
                    const int s = loads % NS;
                    if (loads >= NS && !(ok = all(wait(&sm.empty[s], loads / NS - 1)))) break;
                    if (lane == 0) {
                        umma::mbar_arrive_expect_tx(&sm.full[s], kT);
#pragma unroll
                        for (int c = 0; c < D / 64; ++c)
                            umma::tma_load_2d(skv + s * kT + c * (kTile * 128), (i & 1) ? &tv : &tk, (h * D + 64 * c) * 2,
                                              k0 + (i >> 1) * kTile, &sm.full[s]);
                    }
                    __syncwarp();
                }
                if (lane == 0) umma::mbar_arrive(&sm.uempty[k & 1]);
            }
        } else if (warp == kMmaWarp) {
            constexpr uint32_t id_s = umma::instr_desc(1, 1, kTile, kTile);
            constexpr uint32_t id_o = umma::instr_desc(1, 1, kTile, D) | (1u << 16);      // B is MN-major
            const uint32_t q_addr = umma::smem_addr(sq), kv_addr = umma::smem_addr(skv);
            // the whole warp walks the loop and one lane issues: with the loop inside the lane's branch the
            // descriptors were moved to uniform registers product by product (494 us for 427 at 8192 tokens)
            elected = umma::elect_one();
            int at = 0, seen[2] = {0, 0}, units[2] = {0, 0};            // copies used; key tiles and units of each row tile
            bool ok = !stall || all(wait(&sm.drain, 0));                // (tests: nothing arrives there before the end)
            for (int k = 0; ok; ++k) {
                if (!(ok = all(wait(&sm.ufull[k & 1], k >> 1)))) break;
                const int n = sm.unit[k & 1].n, nt = tiles(sm.unit[k & 1]);
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&sm.uempty[k & 1]);
                if (n < 0) break;
                if (n == 0) continue;
                auto scores = [&](int t, int i) {                       // S_t = Q_t K_i^T
                    const uint64_t ad = desc_k(q_addr + t * kT), bd = desc_k(kv_addr + ((at + 2 * i) % NS) * kT);
                    if (elected) {
#pragma unroll
                        for (int kk = 0; kk < D / 16; ++kk) {
                            const uint32_t step = (uint32_t)((kk >> 2) * (kTile * 128) + (kk & 3) * 32) >> 4;
                            umma::mma_bf16(tmem + kS + t * kTile, ad + step, bd + step, id_s, kk != 0);
                        }
                        umma::mma_commit(&sm.sfull[t]);
                        if (i == n - 1) umma::mma_commit(&sm.qfree[t]);
                    }
                    __syncwarp();
                };
                ok = all(wait(&sm.full[at % NS], at / NS));
                for (int t = 0; t < nt && ok; ++t) {
                    if (!(ok = all(wait(&sm.qfull[t], units[t]++)))) break;
                    umma::fence_after_sync();
                    issued = true;
                    scores(t, 0);
                }
                if (ok && elected) umma::mma_commit(&sm.empty[at % NS]);
                for (int i = 0; i < n && ok; ++i) {
                    const int iv = at + 2 * i + 1, ik = iv + 1;
                    const bool more = i + 1 < n;
                    ok = all(wait(&sm.full[iv % NS], iv / NS));
                    for (int t = 0; t < nt && ok; ++t) {
                        const uint64_t bd = desc_mn(kv_addr + (iv % NS) * kT);
                        for (int half = 0; half < 2 && ok; ++half) {
                            if (!(ok = all(wait(&sm.pfull[t][half], seen[t] + i)))) break;
                            umma::fence_after_sync();
                            if (elected) {
#pragma unroll
                                for (int k4 = 0; k4 < kTile / 32; ++k4) {   // 16 keys: 2 groups of 8 rows
                                    const int kk = half * (kTile / 32) + k4;
                                    umma::mma_bf16_ta(tmem + kO + t * kTile, tmem + kS + t * kTile + kk * 8, bd + (kk * 2048 >> 4), id_o,
                                                      (i | kk) != 0);
                                }
                            }
                        }
                        if (!ok) break;
                        if (elected && t == nt - 1) umma::mma_commit(&sm.empty[iv % NS]);
                        __syncwarp();
                        if (more) {
                            if (t == 0 && !(ok = all(wait(&sm.full[ik % NS], ik / NS)))) break;
                            scores(t, i + 1);
                            if (t == nt - 1 && elected) umma::mma_commit(&sm.empty[ik % NS]);
                        } else {
                            if (elected) umma::mma_commit(&sm.odone[t]);
                        }
                        __syncwarp();
                    }
                }
                at += 2 * n;
                for (int t = 0; t < nt; ++t) seen[t] += n;
            }
        }
    } else {
      asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
      const int t = warp >> 2;
      const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
      const uint32_t ts = tmem + lanes + kS + t * kTile, to = tmem + lanes + kO + t * kTile;
      // a zero scale: as good as zero times any score, and a masked one stays minus infinity
      const float c = a.scale != 0.0f ? a.scale * 1.4426950408889634f : 1.0e-30f;
      const uint64_t cc = f2(c, c);
      int tiles_seen = 0, units_seen = 0;
      bool ok = true;
      for (int k = 0; ok; ++k) {
        if (!(ok = all(wait(&sm.ufull[k & 1], k >> 1)))) break;
        const Unit u = sm.unit[k & 1];
        __syncwarp();
        if (lane == 0) umma::mbar_arrive(&sm.uempty[k & 1]);
        if (u.n < 0) break;
        if (t >= tiles(u)) continue;
        const int n = u.n, h = u.h, q0 = u.q0, k0 = u.k0, off = u.off;
        const int r = (warp & 3) * 32 + lane, pr = a.over_g(r), p_first = u.first + t * per_tile;
        const bool in = pr < per_tile && t * per_tile + pr < u.left;
        const int p = in ? p_first + pr : 0, g = in ? r - pr * G : 0;
        const int lim = in ? p + off : -1;                              // last key seen
        // tiles from here on are masked for some row of the tile
        const int first_masked = p_first + off;
        float m = 0.0f, l = 0.0f, last = 0.0f;                          // reference in log2 units; the last tile's sum
        for (int i = 0; i < n; ++i) {
            if (!(ok = all(wait(&sm.sfull[t], tiles_seen + i)))) break;
            umma::fence_after_sync();
            if (__any_sync(0xffffffffu, last > kGrown)) {               // O_t is complete up to tile i - 1
                const int k = last > kGrown ? (int)(__float_as_uint(last) >> 23) - 127 : 0;
                const float f = __uint_as_float((uint32_t)max(127 - k, 1) << 23);
                m += (float)k;
                l *= f;
#pragma unroll
                for (int x = 0; x < D / 16; ++x) {
                    uint32_t o[16];
                    umma::tmem_ld16(to + 16 * x, o);
                    umma::tmem_ld_wait();
#pragma unroll
                    for (int y = 0; y < 16; ++y) o[y] = __float_as_uint(__uint_as_float(o[y]) * f);
                    umma::tmem_st16(to + 16 * x, o);
                }
            }
            uint32_t s[4][32];
#pragma unroll
            for (int x = 0; x < 4; ++x) umma::tmem_ld32(ts + 32 * x, s[x]);
            umma::tmem_ld_wait();
            if (i * kTile + kTile - 1 > first_masked) {                 // (rows of no position may hold anything)
                const int seen = lim - i * kTile;                       // columns 0 .. seen
                const uint32_t hidden = c < 0.0f ? 0x7F800000u : 0xFF800000u;   // c times it is minus infinity
#pragma unroll
                for (int x = 0; x < 4; ++x)
#pragma unroll
                    for (int y = 0; y < 32; ++y)
                        if (32 * x + y > seen) s[x][y] = hidden;
            }
            if (i == 0) {
                const uint32_t turn = c < 0.0f ? 0x80000000u : 0u;
                auto at = [&](uint32_t v) { return __uint_as_float(v ^ turn); };
                float mx[8];
#pragma unroll
                for (int x = 0; x < 8; ++x) {
                    const uint32_t *v = &s[x >> 1][16 * (x & 1)];
                    mx[x] = fmaxf(at(v[0]), at(v[1]));
#pragma unroll
                    for (int y = 2; y < 16; y += 2) mx[x] = max3(mx[x], at(v[y]), at(v[y + 1]));
                }
                const float top = max3(max3(mx[0], mx[1], mx[2]), max3(mx[3], mx[4], mx[5]), fmaxf(mx[6], mx[7]));
                m = top > -INFINITY ? top * fabsf(c) : 0.0f;
            }
            const uint64_t mm = f2(-m, -m);
            last = 0.0f;
#pragma unroll
            for (int x = 0; x < 2; ++x) {
                uint64_t sum[4] = {0, 0, 0, 0};
                uint32_t w[32];
#pragma unroll
                for (int y = 0; y < 32; ++y) {
                    const uint64_t d = fma2(f2(__uint_as_float(s[2 * x + (y >> 4)][(2 * y) & 31]), __uint_as_float(s[2 * x + (y >> 4)][(2 * y + 1) & 31])), cc, mm);
                    const float p0 = ex2(lo32(d)), p1 = ex2(hi32(d));
                    sum[y & 3] = add2(sum[y & 3], f2(p0, p1));
                    w[y] = pack_bf16(p0, p1);
                }
                umma::tmem_st32(ts + 32 * x, w);
                sum[0] = add2(add2(sum[0], sum[1]), add2(sum[2], sum[3]));
                last += lo32(sum[0]) + hi32(sum[0]);
                umma::tmem_st_wait();
                umma::fence_before_sync();
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&sm.pfull[t][x]);   // (a thread each: the arrivals queue up)
            }
            l += last;
            if (!in) last = 0.0f;
        }
        // ---- epilogue: o = O / l ----
        if (ok && n > 0) ok = all(wait(&sm.odone[t], units_seen));
        tiles_seen += n;
        units_seen += n > 0;
        if (ok) {
            umma::fence_after_sync();
            const size_t at = (size_t)(q0 + p) * a.ldo + (size_t)(h * G + g) * D;     // this row's place in o
            const float inv = lim >= 0 ? 1.0f / l : 0.0f;
            const uint64_t inv2 = f2(inv, inv);
            if (l != l && m < INFINITY) l = -1.0f;                      // a score is NaN, and so is all of the row
            const uint32_t keep = lim >= 0 ? 0xFFFFFFFFu : 0u;
            uint64_t zero = 0;                                          // NaN from where some value is not finite
            const uint32_t inside = __ballot_sync(0xffffffffu, in);
            uint8_t *buf = so + warp * (32 * 128);
#pragma unroll
            for (int x = 0; x < D / 64; ++x) {
                // 64 values of each row through shared memory, so that eight lanes write one row's 128 bytes (rows
                // written by their own threads: 32 places per store)
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    uint32_t o[32], w[16];
                    if (n > 0) {
                        umma::tmem_ld32(to + 64 * x + 32 * y, o);
                        umma::tmem_ld_wait();
                    }
#pragma unroll
                    for (int z = 0; z < 16; ++z) {
                        const uint64_t v = mul2(f2(__uint_as_float(o[2 * z]), __uint_as_float(o[2 * z + 1])), inv2);
                        zero = fma2(v, 0, zero);
                        w[z] = pack_bf16(lo32(v), hi32(v)) & keep;
                    }
#pragma unroll
                    for (int z = 0; z < 4; ++z)
                        *reinterpret_cast<uint4 *>(buf + lane * 128 + (((4 * y + z) ^ (lane & 7)) << 4)) =
                            make_uint4(w[4 * z], w[4 * z + 1], w[4 * z + 2], w[4 * z + 3]);
                }
                __syncwarp();
#pragma unroll
                for (int z = 0; z < 8; ++z) {
                    const int row = 4 * z + (lane >> 3), ch = lane & 7;
                    const uint4 v = *reinterpret_cast<const uint4 *>(buf + row * 128 + ((ch ^ (row & 7)) << 4));
                    const size_t dst = __shfl_sync(0xffffffffu, at, row);
                    if (inside >> row & 1) *reinterpret_cast<uint4 *>(a.o + dst + 64 * x + 8 * ch) = v;
                }
                __syncwarp();
            }
            const bool fine = lim < 0 || (l > 0.0f && l < INFINITY && lo32(zero) + hi32(zero) == 0.0f);
            const uint32_t again = __ballot_sync(0xffffffffu, in && !fine);
            if (again) rows_again<D>(a, h, q0, k0, off, p, g, l, again);
        }
      }
    }

    // after a timeout: copies and products in flight finish (bounded) before
    // the memory is released
    __syncthreads();
    if (sm.timeout) {
        if (warp == kTmaWarp && lane == 0)
            for (int i = max(0, loads - NS); i < loads; ++i)
                umma::mbar_wait(&sm.full[i % NS], (uint32_t)((i / NS) & 1), kWaitLimit);
        if (warp == kUnitWarp && lane == 0)
            for (int t = 0; t < 2; ++t)
                if (sm.q_count[t] > 0) umma::mbar_wait(&sm.qfull[t], (uint32_t)((sm.q_count[t] - 1) & 1), kWaitLimit);
        if (warp == kMmaWarp && elected && issued) {
            umma::mma_commit(&sm.drain);
            umma::mbar_wait(&sm.drain, 0, kWaitLimit);
        }
        if (tid == 0) flag(a.st, QSPEC_ERR_TIMEOUT);
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) umma::tmem_free(tmem, kCols);
}

template <int D>
int launch(const Args &a, cudaStream_t stream, uint32_t wait_limit, int stall) {
    const long long units = (long long)a.q_rows / (kTile / a.G) + a.B;      // at most, of one tile
    if (units * a.H >= (1LL << 31)) return QSPEC_ERR_SHAPE;
    // no key rows: no copy is issued, and the maps only have to be valid
    const bool none = a.k_rows == 0;
    CUtensorMap tk, tv;
    const int cols = (none ? a.H * a.G : a.H / a.share) * D * 2;
    if (byte_tmap_sw128(&tk, none ? a.q : a.k, none ? a.q_rows : a.k_rows, cols, (size_t)(none ? a.ldq : a.ldk) * 2, kTile) ||
        byte_tmap_sw128(&tv, none ? a.q : a.v, none ? a.q_rows : a.k_rows, cols, (size_t)(none ? a.ldq : a.ldv) * 2, kTile))
        return QSPEC_ERR_UNSUPPORTED;
    CUtensorMap tq;
    if (row_box_tmap_sw128(&tq, a.q, D * 2, a.H * a.G, a.q_rows, (size_t)a.ldq * 2, a.G, kTile / a.G)) return QSPEC_ERR_UNSUPPORTED;
    auto kern = attn_prompt_kernel<D>;
    int rc = smem_limit_once(reinterpret_cast<const void *>(kern), (int)smem_total<D>());
    if (rc) return rc;
    return launch_pdl("qspec_attn_prompt", kern, dim3((unsigned)std::min<long long>(sm_count(), units * a.H)), dim3(kThreads), smem_total<D>(), stream, tq,
                      tk, tv, a, wait_limit, stall);
}

}  // namespace apr

}  // namespace

}  // namespace qspec

using namespace qspec;

extern "C" int qspec_debug_attn_prompt_bounded(const uint16_t *q_bf16, int ldq, const uint16_t *k_bf16, int ldk,
                                               const uint16_t *v_bf16, int ldv, const int32_t *q_start,
                                               const int32_t *k_start, int q_rows, int k_rows, int B, int Hq, int H, int D,
                                               float scale, uint16_t *o_bf16, int ldo, uint32_t wait_limit, int stall,
                                               int32_t *dev_status, qspec_stream_t stream) {
    if (!q_start || !k_start || (q_rows > 0 && (!q_bf16 || !o_bf16)) || (k_rows > 0 && (!k_bf16 || !v_bf16)))
        return QSPEC_ERR_NULL;
    if (q_rows < 0 || k_rows < 0 || B < 1 || H < 1 || Hq < H || Hq % H || Hq > 65535 || (D != 64 && D != 128) ||
        !std::isfinite(scale) || ldq < (long long)Hq * D || ldo < (long long)Hq * D || ldk < (long long)H * D ||
        ldv < (long long)H * D || wait_limit < 1)
        return QSPEC_ERR_SHAPE;
    if ((ldq | ldk | ldv | ldo) % 8 || !aligned(q_bf16, 16) || !aligned(k_bf16, 16) || !aligned(v_bf16, 16) ||
        !aligned(o_bf16, 16) || !aligned(q_start, 4) || !aligned(k_start, 4))
        return QSPEC_ERR_ALIGN;
    int rc = check_device();
    if (rc || q_rows == 0) return rc;
    // heads to a row tile: all of a KV head's up to 128, else the largest equal part
    int G = Hq / H, share = 1;
    while (G / share > apr::kTile || G % share) ++share;
    G /= share;
    const apr::Args a{q_bf16, k_bf16, v_bf16, q_start, k_start, o_bf16, dev_status, ldq, ldk, ldv, ldo, q_rows, k_rows, B,
                      H * share, G, share, G == 1 ? 0u : (uint32_t)((1ull << 32) / G + 1), scale};
    return D == 128 ? apr::launch<128>(a, as_cuda(stream), wait_limit, stall)
                    : apr::launch<64>(a, as_cuda(stream), wait_limit, stall);
}

extern "C" int qspec_attn_prompt(const uint16_t *q_bf16, int ldq, const uint16_t *k_bf16, int ldk,
                                 const uint16_t *v_bf16, int ldv, const int32_t *q_start, const int32_t *k_start,
                                 int q_rows, int k_rows, int B, int Hq, int H, int D, float scale, uint16_t *o_bf16,
                                 int ldo, int32_t *dev_status, qspec_stream_t stream) {
    return qspec_debug_attn_prompt_bounded(q_bf16, ldq, k_bf16, ldk, v_bf16, ldv, q_start, k_start, q_rows, k_rows, B, Hq,
                                           H, D, scale, o_bf16, ldo, kWaitLimit, 0, dev_status, stream);
}
