// fp8_block_tile.cu -- products of E4M3 codes with a scale for each block of 128
// for many tokens (prompts, verify passes of large batches): the linear, and the gated
// product.  Definitions: fp8_block_stream.cu.
//
// A CTA takes 128 tokens (the accumulator's lanes) x 256 channels (its columns; gated: 128
// of the gate, 128 of the up projection).  Persistent: it goes through tiles in groups of
// 8 token tiles, whose operands stay in L2 while the channels go by.
// The tensor cores cannot scale a block's sums, so the products of a block (K = 128)
// go into an accumulator of their own, two of them in turn (all of tensor memory), and
// eight warps (thread = token, half the channels) add it to 128 sums in registers, times
// the token's scale and the channels', while the next block's products run.  The sums' way out
// (SiLU, product, maxima, codes) has two blocks' products of the next tile beside it.
// One warp issues the copies, one the products, one fetches the scales some blocks ahead.
// A block counts its sum times s = (token's scale x channels'), s rounded to fp32: where that is subnormal digits are lost
// (include/qspec.h says how many).  Multiplying by the two one after another there, as forms of this loop did that had to
// look for such blocks, took 4 to 10 % of every call, whichever warp looked.
// The tiles behind the last full round of CTAs are split along K over the CTAs of a
// cluster, whose parts meet in shared memory, in the order of K.
//
// Bound: shared memory, by count.  A block is written (48 KB) and read by the products (48 KB), 768
// clocks at 128 bytes; the products take 512, the packed additions 256.  Measured: some 830
// clocks a block (0.43 us), 8192 x 4096 x 14336 in 354 us (2720 TFLOP/s), gated 8192 x 14336 x
// 4096 in 715 us (2690) as long as the clock holds, 410 and 811 us under the power cap (1.6 GHz).
// The same pipeline without the additions, one accumulator handed over for 16 blocks: 317 and 630.
// The counters of the memory's banks agree with the bytes (13.5 K words read and 13.4 K written a block, of
// which 12.3 K each are the operands'), but not on the rate: they take 64 words a clock of either kind for the peak.
// Pairs of CTAs (256 tokens, half of either operand in each) need 512 clocks of shared memory,
// but with barriers in the other CTA an accumulator's way round took 900: 363 us, with sixteen
// warps of 64 sums 374, and at 80 to 512 tokens a half-empty tile more often (gated 128 x
// 14336 x 4096 36 us for 25).  Halves of 128 columns with two accumulators each read the tokens
// twice: 477 us.
#include <algorithm>
#include <climits>

#include "fp8_block_host.h"
#include "umma.cuh"

namespace qspec {

namespace {

namespace f8t {

using f8b::add2;
using f8b::Args;
using f8b::desc_sw128;
using f8b::f2;
using f8b::fma2;
using f8b::hi32;
using f8b::kMaxSplit;
using f8b::lo32;
using f8b::max_abs;
using f8b::mul2;

constexpr int kRows = 128, kCols = 256;              // of the accumulator
constexpr int kWorkWarps = 8, kWork = 32 * kWorkWarps, kLoadWarp = 8, kMmaWarp = 9, kScaleWarp = 10, kThreads = kWork + 128;
constexpr int kPiece = 128 * 128;                    // 128 rows of an operand's block
constexpr int kStage = 3 * kPiece, kStages = 4;
static_assert(kStages >= 2, "a stage's products must not be done twice before all warps have looked: two accumulators");
static_assert(kRows * kCols * 4 <= kStages * kStage, "a CTA's sums lie over the stages");
constexpr int kBatch = 4, kBatches = 4;              // scales: blocks per hand-over, hand-overs in flight
constexpr int kGroupTiles = 8;                       // token tiles that go through the channels together
// registers per thread: all start with 168; 128 sums and their operands need more, the issuing warps less (shares at
// which either kernel compiles without spills: 200 / 104 cost the gated one 10 %)
template <bool kGated>
struct Regs {
    static constexpr int kWork = kGated ? 216 : 208, kRest = kGated ? 72 : 88;
    static_assert(kThreads * 168 <= 65536 && f8t::kWork * kWork + 128 * kRest <= kThreads * 168, "register shares");
};

struct Ctl {
    uint64_t full[kStages], done[kStages];           // a stage's copies landed; its products done: stage free, sums there
    uint64_t acc_empty[2];
    uint64_t scale_full[kBatches], scale_empty[kBatches];
    uint64_t drain;
    uint32_t tmem;
    int timeout;
    float token_scale[kBatches * kBatch][kRows], weight_scale[kBatches * kBatch][2];
    float top[2][2][kRows];                          // gated: maxima of the two halves of the channels, two tiles' in turn
};
constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + sizeof(Ctl), kSmemApart = kSmem + kWorkWarps * 32 * 17 * 4;

// What a launch goes through: the tiles 0 .. full - 1 one by one, each CTA every gridDim.x-th, then the others in parts
// of K, `split` CTAs of a cluster to a tile.
struct Plan {
    int row_tiles, col_tiles, full, split;
};

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float min_of(float a, float b, float c) {           // keeps a NaN
    float d;
    asm("min.NaN.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
    return d;
}
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

// A warp's part of shared memory for results whose rows begin anywhere (17: the rows of it begin in different banks).
struct Rows {
    uint32_t w[32][17];
};

// 32 neighbouring channels n .. n + 31 of a row m to bf16, thread = row.  In 16-byte stores, or 32-byte ones where y allows
// (`wide`; half the way through the store unit, which a warp's 32 rows take one by one); kApart: through shared
// memory, row after row, lane = channel (8192 x 4097 x 256 in 43 us; value by value from where they are 278).
template <bool kApart>
__device__ __forceinline__ void store_row(const Args &a, int m, int n, bool wide, const uint64_t *v, Rows *buf) {
    if constexpr (kApart) {
        const int lane = threadIdx.x & 31, m0 = m - lane;
#pragma unroll
        for (int j = 0; j < 16; ++j) buf->w[lane][j] = pack_bf16(lo32(v[j]), hi32(v[j]));
        __syncwarp();
        if (n + lane < a.N)
#pragma unroll 8
            for (int r = 0; r < 32; ++r)
                if (m0 + r < a.M) a.y[(size_t)(m0 + r) * a.ldy + n + lane] = reinterpret_cast<const uint16_t *>(buf->w[r])[lane];
        __syncwarp();
    } else if (m < a.M) {
        uint16_t *row = a.y + (size_t)m * a.ldy;
#pragma unroll
        for (int j = 0; j < 16; j += 8) {
            const int at = n + 2 * j;
            if (at + 16 <= a.N) {
                uint32_t w[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) w[e] = pack_bf16(lo32(v[j + e]), hi32(v[j + e]));
                f8b::store32(row + at, w, wide);
            } else {
#pragma unroll
                for (int e = 0; e < 16; ++e)
                    if (at + e < a.N) row[at + e] = float_to_bf16_bits(e % 2 == 0 ? lo32(v[j + e / 2]) : hi32(v[j + e / 2]));
            }
        }
    }
}

template <bool kGated, bool kApart>
__global__ void __launch_bounds__(kThreads, 1)
    tile_kernel(const __grid_constant__ CUtensorMap t0, const __grid_constant__ CUtensorMap t1,
                const __grid_constant__ CUtensorMap tx, const __grid_constant__ Args a, const Plan plan, bool wide_y,
                bool wide_h, uint32_t wait_limit, int stall) {
    constexpr int kChannels = kGated ? 128 : 256;                // channels of a tile
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stages = smem_raw + ((1024u - (umma::smem_addr(smem_raw) & 1023u)) & 1023u);
    Ctl &sm = *reinterpret_cast<Ctl *>(stages + (size_t)kStages * kStage);
    Rows *rows = reinterpret_cast<Rows *>(&sm + 1);              // (kApart)
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int G = a.K / kGroup, cta = (int)blockIdx.x, ctas = (int)gridDim.x;
    const int fulls = cta < plan.full ? (plan.full - cta + ctas - 1) / ctas : 0;      // whole tiles of this CTA
    const int part = cta % plan.split;                            // of K, of its last tile
    const int last = plan.full + cta / plan.split;
    const int items = fulls + (last < plan.row_tiles * plan.col_tiles ? 1 : 0);
    const bool shared = items > fulls;
    const int shared_k0 = (int)((long long)G * part / plan.split), shared_nk = (int)((long long)G * (part + 1) / plan.split) - shared_k0;
    // item i: its tile's place (token tile, channel tile) and blocks of K
    auto item = [&](int i, int &rt, int &ct, int &k0) -> int {
        const int t = i < fulls ? cta + i * ctas : last;
        const int in = kGroupTiles * plan.col_tiles, g = t / in, r = t - g * in;
        const int rows = min(kGroupTiles, plan.row_tiles - g * kGroupTiles);
        ct = rows == kGroupTiles ? r / kGroupTiles : r / rows;
        rt = g * kGroupTiles + (r - ct * rows);
        k0 = i < fulls ? 0 : shared_k0;
        return i < fulls ? G : shared_nk;
    };
    volatile int *timeout = &sm.timeout;
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (umma::mbar_try_wait(bar, parity & 1)) return true;
        if (*timeout) return false;
        if (umma::mbar_wait(bar, parity & 1, wait_limit)) return true;
        *timeout = 1;
        return false;
    };
    auto all = [](bool mine) { return __all_sync(0xffffffffu, mine) != 0; };
    // where four neighbouring sums of a token lie while the parts of K meet
    auto piece = [&](int row, int p) { return reinterpret_cast<float4 *>(stages) + row * (kCols / 4) + (p ^ (row & 7)); };
    auto load_weights = [&](int s, int g, int n0) {               // block g of K, channels n0 ..., into stage s
        uint8_t *at = stages + (size_t)s * kStage;
        umma::mbar_arrive_expect_tx(&sm.full[s], kStage);
        umma::tma_load_2d(at + kPiece, &t0, g * kGroup, n0, &sm.full[s]);
        umma::tma_load_2d(at + 2 * kPiece, kGated ? &t1 : &t0, g * kGroup, n0 + (kGated ? 0 : 128), &sm.full[s]);
    };
    auto load_tokens = [&](int s, int g, int m0) {
        umma::tma_load_2d(stages + (size_t)s * kStage, &tx, g * kGroup, m0, &sm.full[s]);
    };

    const bool elected = umma::elect_one();
    int early = 0;                                                // blocks of the first tile whose weights are under way
    if (warp == kLoadWarp) {
        int rt, ct, k0;
        const int nk = items > 0 ? item(0, rt, ct, k0) : 0;
        early = min(kStages, nk);
        if (elected) {
            sm.timeout = 0;
            for (int i = 0; i < kStages; ++i) {
                umma::mbar_init(&sm.full[i], 1);
                umma::mbar_init(&sm.done[i], 1);
            }
            for (int i = 0; i < 2; ++i) umma::mbar_init(&sm.acc_empty[i], kWorkWarps);
            for (int i = 0; i < kBatches; ++i) {
                umma::mbar_init(&sm.scale_full[i], 1);
                umma::mbar_init(&sm.scale_empty[i], kWorkWarps);
            }
            umma::mbar_init(&sm.drain, 1);
            umma::mbar_fence_init();
            umma::fence_proxy_async();
            umma::fence_proxy_async_global();           // (the weights may be the kernel's in front, which is complete)
            // the first stages' weights at once, before the dependency wait too
            for (int i = 0; i < early; ++i) load_weights(i, k0 + i, ct * kChannels);
        }
        __syncwarp();
    }
    if (warp == kMmaWarp) umma::tmem_alloc(&sm.tmem, 2 * kCols);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    pdl_launch_dependents();
    const uint32_t tmem = sm.tmem;
    int loads = 0, issued = 0;                                    // blocks whose copies, whose products were issued
    auto meet = [&]() {                                           // (behind the CTA's own barrier and a timeout's drain)
        if (plan.split > 1)
            umma::cluster_sync();
        else
            __syncthreads();
    };

    if (warp >= kWorkWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(Regs<kGated>::kRest));
        // (the issuing warps go through their loops whole and elect a lane where it counts: a lane's own loop is
        // slower by the divergence that the compiler allows for at every step)
        if (warp == kLoadWarp) {
            pdl_wait();
            bool ok = true;
            int s = 0, turn = 0;                                  // the stage, and how often it was filled before
            for (int i = 0; i < items && ok; ++i) {
                int rt, ct, k0;
                const int nk = item(i, rt, ct, k0);
                for (int g = k0; g < k0 + nk; ++g) {
                    if (!(ok = turn == 0 || all(wait(&sm.done[s], (uint32_t)(turn + 1))))) break;
                    if (elected) {
                        if (loads >= early) load_weights(s, g, ct * kChannels);
                        load_tokens(s, g, rt * kRows);
                    }
                    __syncwarp();
                    ++loads;
                    if (++s == kStages) {
                        s = 0;
                        ++turn;
                    }
                }
            }
        } else if (warp == kMmaWarp) {
            constexpr uint32_t idesc = umma::instr_desc(0, 0, kRows, kCols);                 // e4m3 x e4m3 -> f32
            const int blocks = fulls * G + (shared ? shared_nk : 0);
            int s = 0;
            uint32_t turn = 0;
            pdl_wait();
            const bool go = !stall || all(wait(&sm.drain, 0));   // (tests: nothing arrives there before the end)
            for (; go && issued < blocks; ++issued) {
                const int b = issued & 1;
                if (!all(wait(&sm.full[s], turn)) || !all(wait(&sm.acc_empty[b], (uint32_t)(issued / 2 + 1)))) break;
                umma::fence_after_sync();
                const uint32_t at = umma::smem_addr(stages + (size_t)s * kStage);
                const uint64_t ad = desc_sw128(at), bd = desc_sw128(at + kPiece);
                if (elected) {
#pragma unroll
                    for (int kk = 0; kk < kGroup / 32; ++kk)      // K = 32 bytes per MMA: +2 in the address field
                        umma::mma_e4m3(tmem + b * kCols, ad + 2 * kk, bd + 2 * kk, idesc, kk != 0 ? 1u : 0u);
                    umma::mma_commit(&sm.done[s]);
                }
                __syncwarp();
                if (++s == kStages) {
                    s = 0;
                    ++turn;
                }
            }
        } else if (warp == kScaleWarp) {
            // the blocks' scales, some way ahead of the work (a load from L2 takes as long as two blocks); coherent loads,
            // past L1, as the kernel in front may write them while this one is resident
            const int blocks_n = (a.N + kGroup - 1) / kGroup;
            int i = 0, g = 0, rt, ct, k0, nk = 0;
            if (items > 0) nk = item(0, rt, ct, k0);
            pdl_wait();
            for (int base = 0; i < items; base += kBatch) {
                float x[kBatch][kRows / 32], w[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const bool some = i < items;
                    const int m0 = rt * kRows + lane;
#pragma unroll
                    for (int e = 0; e < kRows / 32; ++e)
                        x[u][e] = some && m0 + 32 * e < a.M ? __ldcg(a.sa + (size_t)(k0 + g) * a.lds + m0 + 32 * e) : 0.0f;
                    // lane 0: of the lower 128 channels, or the gate; lane 1: of the upper 128, or up
                    const float *from = kGated && lane == 1 ? a.s1 : a.s0;
                    w[u] = some && lane < 2 ? __ldcg(from + (size_t)(kGated ? ct : min(2 * ct + lane, blocks_n - 1)) * G + k0 + g) : 0.0f;
                    if (some && ++g == nk) {
                        g = 0;
                        if (++i < items) nk = item(i, rt, ct, k0);
                    }
                }
                const int slot = base / kBatch % kBatches;
                if (!all(wait(&sm.scale_empty[slot], (uint32_t)(base / (kBatch * kBatches) + 1)))) break;
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
#pragma unroll
                    for (int e = 0; e < kRows / 32; ++e) sm.token_scale[slot * kBatch + u][lane + 32 * e] = x[u][e];
                    if (lane < 2) sm.weight_scale[slot * kBatch + u][lane] = w[u];
                }
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&sm.scale_full[slot]);
            }
        }
        // after a timeout: the copies and products in flight finish (bounded) before the memory they use is used
        // again; both issuers stopped at the timeout, so at most kStages copies are outstanding
        __syncthreads();
        if (*timeout) {
            if (warp == kLoadWarp && elected)
                for (int b = max(0, loads - kStages); b < loads; ++b)
                    umma::mbar_wait(&sm.full[b % kStages], (uint32_t)((b / kStages) & 1), kWaitLimit);
            if (warp == kMmaWarp && elected && issued > 0) {
                umma::mma_commit(&sm.drain);
                umma::mbar_wait(&sm.drain, 0, kWaitLimit);
            }
            if (warp == kScaleWarp && lane == 0) flag(a.st, QSPEC_ERR_TIMEOUT);
            __syncwarp();
        }
        // (freed before the cluster's barrier: a CTA that waits for its peers holds no tensor memory that one of them may
        // be waiting for, behind another stream's kernel)
        umma::fence_after_sync();
        if (warp == kMmaWarp) umma::tmem_free(tmem, 2 * kCols);
        meet();
        if (plan.split > 1) umma::cluster_sync();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(Regs<kGated>::kWork));
        // ---- thread = token; warps 0 .. 3 the lower half of the channels (gated: of both parts), 4 .. 7 the upper ----
        const int half = warp >> 2, row = 32 * (warp & 3) + lane;
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        // columns of its four chunks of 32
        auto column = [&](int c) { return kGated ? (c >> 1) * 128 + half * 64 + (c & 1) * 32 : half * 128 + c * 32; };
        int done = 0, parity = 0;
        pdl_wait();
        for (int i = 0; i < items; ++i) {
            int rt, ct, k0;
            const int nk = item(i, rt, ct, k0), m = rt * kRows + row;
            const bool in = m < a.M;
            uint64_t acc[4][16];
#pragma unroll
            for (int c = 0; c < 4; ++c)
#pragma unroll
                for (int j = 0; j < 16; ++j) acc[c][j] = 0;
            bool ok = true;
            for (int g = 0; g < nk; ++g) {
                const int b = done & 1, at = done % (kBatch * kBatches), slot = at / kBatch;
                if (at % kBatch == 0 && !all(wait(&sm.scale_full[slot], (uint32_t)(done / (kBatch * kBatches))))) ok = false;
                const float x = sm.token_scale[at][row];
                const float s0 = x * sm.weight_scale[at][kGated ? 0 : half], s1 = kGated ? x * sm.weight_scale[at][1] : s0;
                if (!(ok = ok && all(wait(&sm.done[done % kStages], (uint32_t)(done / kStages))))) break;
                umma::fence_after_sync();
                // a chunk is on its way while the one before it is added
                uint32_t d[2][32];
                umma::tmem_ld32(tmem + lanes + b * kCols + column(0), d[0]);
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                    umma::tmem_ld_wait();
                    if (c < 3) umma::tmem_ld32(tmem + lanes + b * kCols + column(c + 1), d[(c + 1) & 1]);
                    if (c == 3) {
                        umma::fence_before_sync();
                        __syncwarp();
                        if (lane == 0) {
                            umma::mbar_arrive(&sm.acc_empty[b]);
                            if (at % kBatch == kBatch - 1) umma::mbar_arrive(&sm.scale_empty[slot]);
                        }
                    }
                    const uint64_t s = c < 2 ? f2(s0, s0) : f2(s1, s1);
#pragma unroll
                    for (int j = 0; j < 16; ++j)
                        acc[c][j] = fma2(f2(__uint_as_float(d[c & 1][2 * j]), __uint_as_float(d[c & 1][2 * j + 1])), s, acc[c][j]);
                }
                ++done;
            }
            // ---- the sums' way out (after a timeout too, without stores: the warps meet in it) ----
            if (i == fulls) {
                // [token][256 columns] over the stages, whose products are done; 16-byte pieces exchanged within 128 bytes
                // by the token, for the banks
                if (ok) {
#pragma unroll
                    for (int c = 0; c < 4; ++c)
#pragma unroll
                        for (int j = 0; j < 16; j += 2)
                            *piece(row, column(c) / 4 + j / 2) =
                                make_float4(lo32(acc[c][j]), hi32(acc[c][j]), lo32(acc[c][j + 1]), hi32(acc[c][j + 1]));
                }
            } else if constexpr (!kGated) {
                if (ok) {
#pragma unroll
                    for (int c = 0; c < 4; ++c) store_row<kApart>(a, m, ct * kChannels + column(c), wide_y, acc[c], rows + warp);
                }
            } else {
                // h = g u / (1 + exp(-g)), two quotients from one reciprocal 1 / (a b) where no gate of the thread's is so
                // low that the product passes fp32: the reciprocals and exponentials bound this part
                constexpr float kLog2e = 1.4426950408889634f;
                float low = 0.0f, amax = 0.0f;
#pragma unroll
                for (int c = 0; c < 2; ++c)
#pragma unroll
                    for (int j = 0; j < 16; ++j) low = min_of(low, lo32(acc[c][j]), hi32(acc[c][j]));
                if (low >= -43.0f) {                             // (no NaN)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const uint64_t x = mul2(acc[c][j], f2(-kLog2e, -kLog2e));
                            const uint64_t e = add2(f2(ex2(lo32(x)), ex2(hi32(x))), f2(1.0f, 1.0f));
                            const float r = rcp_approx(lo32(e) * hi32(e));
                            const uint64_t v = mul2(mul2(acc[c][j], mul2(f2(hi32(e), lo32(e)), f2(r, r))), acc[c + 2][j]);
                            amax = max_abs(amax, lo32(v), hi32(v));
                            acc[c][j] = v;
                        }
                } else {
#pragma unroll
                    for (int c = 0; c < 2; ++c)
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float v0 = f8b::gated(lo32(acc[c][j]), lo32(acc[c + 2][j]));
                            const float v1 = f8b::gated(hi32(acc[c][j]), hi32(acc[c + 2][j]));
                            amax = max_abs(amax, v0, v1);
                            acc[c][j] = f2(v0, v1);
                        }
                }
                sm.top[parity][half][row] = amax;
                asm volatile("bar.sync %0, 64;" ::"r"(1 + (warp & 3)) : "memory");      // (the two warps of the same tokens)
                amax = max_abs(amax, sm.top[parity][half ^ 1][row], 0.0f);
                parity ^= 1;
                const int n = ct * kChannels + half * 64;
                if (ok && a.y != nullptr) {
#pragma unroll
                    for (int c = 0; c < 2; ++c) store_row<kApart>(a, m, n + c * 32, wide_y, acc[c], rows + warp);
                }
                if (in && ok) {
                    if (a.hq != nullptr) {
                        const f8b::Quant q(amax);
                        const uint64_t by = f2(q.inv, q.inv);
                        if (q.up != 1.0f) {                              // (h in bf16 was stored before; no code of -0 for a scale of 0)
#pragma unroll
                            for (int c = 0; c < 2; ++c)
#pragma unroll
                                for (int j = 0; j < 16; ++j) acc[c][j] = q.s == 0.0f ? 0 : mul2(acc[c][j], f2(q.up, q.up));
                        }
                        uint8_t *out = a.hq + (size_t)m * a.N + n;
#pragma unroll
                        for (int c = 0; c < 2; ++c) {
                            uint32_t w[8];
#pragma unroll
                            for (int e = 0; e < 8; ++e) {
                                const uint64_t v0 = mul2(acc[c][2 * e], by), v1 = mul2(acc[c][2 * e + 1], by);
                                w[e] = f8b::codes4(lo32(v0), hi32(v0), lo32(v1), hi32(v1));
                            }
                            f8b::store32(out + 32 * c, w, wide_h);
                        }
                        if (half == 0) a.sh[(size_t)ct * a.ldh + m] = q.s;
                    }
                    if (half == 0 && !(amax < (a.y != nullptr ? 3.3961775292304601e38f : INFINITY))) flag(a.st, QSPEC_ERR_NONFINITE);
                }
            }
        }
        __syncthreads();
        meet();
        if (shared) {
            // ---- the parts of K meet: a warp takes a token, its lanes four channels of either half ----
            int rt, ct, k0;
            item(fulls, rt, ct, k0);
            const int m0 = rt * kRows, tokens = min(kRows, a.M - m0);
            // 0, as the parts are the cluster's CTAs in their order; as a number that the compiler does not know it keeps the
            // peers' addresses out of registers in front of the loop (gated 192 x 14336 x 4096 33.2 us, with a plain 0 33.9)
            const int first = (int)umma::cluster_rank() - part;
            const int r0 = warp * plan.split + part, step = kWorkWarps * plan.split;
            const auto sums = [&](int r, int half) { return reinterpret_cast<const float *>(piece(r, 32 * half + lane)); };
            const auto store = [&](int r, const float (&v0)[4], const float (&v1)[4]) {
                f8b::store_bf16(a, m0 + r, ct * kChannels + 4 * lane, v0);
                f8b::store_bf16(a, m0 + r, ct * kChannels + 128 + 4 * lane, v1);
            };
            // Few parts and plain sums: two tokens at a time, 1.7 us less at 512 x 4096 x 4096 (16.5 us to 14.8).  More parts
            // fill the registers with one token; behind the gate two cost the kernel's loop 2 to 3 % by what the compiler
            // made of it, and won nothing.
            if (!kGated && plan.split <= 4) {
                for (int r = r0; r < tokens; r += 2 * step) {
                    const int next = min(r + step, tokens - 1);
                    const float *at[4] = {sums(r, 0), sums(r, 1), sums(next, 0), sums(next, 1)};
                    float v[4][4];
                    f8b::sum_parts<4>(at, plan.split, first, v);
                    store(r, v[0], v[1]);
                    if (r + step < tokens) store(next, v[2], v[3]);
                }
            } else {
                for (int r = r0; r < tokens; r += step) {
                    const float *at[2] = {sums(r, 0), sums(r, 1)};
                    float v[2][4];
                    f8b::sum_parts(at, plan.split, first, v);
                    if constexpr (kGated) f8b::store_gated(a, m0 + r, ct, lane, v[0], v[1]);
                    else store(r, v[0], v[1]);
                }
            }
        }
        if (plan.split > 1) umma::cluster_sync();                // (a peer may still read this CTA's sums)
    }
}

template <bool kGated>
struct Kernel {
    static const void *address() { return reinterpret_cast<const void *>(tile_kernel<kGated, false>); }
    static constexpr int threads = kThreads, per = 1;
    static constexpr size_t smem = kSmem;
    static constexpr bool carveout = false;
};

template <bool kGated, bool kApart>
int launch(const char *where, const uint8_t *xq, const uint8_t *w0, const uint8_t *w1, const Args &a, cudaStream_t stream,
           uint32_t wait_limit, int stall) {
    CUtensorMap t0, t1, tx;
    if (byte_tmap_sw128(&t0, w0, a.N, a.K, (size_t)a.K, 128) || (kGated && byte_tmap_sw128(&t1, w1, a.N, a.K, (size_t)a.K, 128)) ||
        byte_tmap_sw128(&tx, xq, a.M, a.K, (size_t)a.K, 128))
        return QSPEC_ERR_UNSUPPORTED;
    if (!kGated) t1 = t0;
    auto kern = tile_kernel<kGated, kApart>;
    constexpr size_t smem = kApart ? kSmemApart : kSmem;
    int rc = smem_limit_once(reinterpret_cast<const void *>(kern), (int)smem);
    if (rc) return rc;
    constexpr int kChannels = kGated ? 128 : 256;
    Plan plan = {(a.M + kRows - 1) / kRows, (a.N + kChannels - 1) / kChannels, 0, 1};
    const long long all = (long long)plan.row_tiles * plan.col_tiles;
    if (all > INT_MAX / 16) return QSPEC_ERR_SHAPE;
    const int tiles = (int)all, G = a.K / kGroup;
    // The cluster's size by what a call would take, in blocks of K of one CTA: full rounds of tiles, then the rest in as
    // many parts as there are CTAs for; the parts' meeting costs some blocks too, more behind the gate, and in two parts
    // with no round before them more again (the whole tiles have the machine's memory for fewer CTAs).  One part / several, us:
    // linear 512 x 4096 (64 tiles) with K = 2048 11.1 / 11.3, 2560 12.7 / 12.1, 4096 17.6 / 14.6; 256 x 4096 (in four) 1536
    // 8.9 / 9.8, 2048 10.6 / 10.4; gated 128 x 8192 (64 tiles) 2048 11.7 / 15.1, 4096 18.9 / 20.2; 192 x 14336 (224 tiles, the last
    // 72 in two) 2048 19.5 / 22.0, 4096 33.5 / 32.7; 128 x 4096 (in four) 1536 8.8 / 10.4.
    const f8b::Resident there = f8b::resident<Kernel<kGated>>();
    double least = 1e30;
    int c = 1, grid = 0;
    for (int s = 1; s <= kMaxSplit && s <= G; ++s) {
        const int ctas = there.ctas[s];
        if (ctas < s) continue;
        const int rounds = tiles / ctas, rest = tiles - rounds * ctas;
        if (s > 1 && (rest == 0 || rest * s > ctas)) continue;
        const double meet = kGated ? (s == 2 && rounds == 0 ? 18.0 : 13.0) : s == 2 ? 8.5 : 11.0;
        const double takes = (double)rounds * G + (rest == 0 ? 0.0 : s == 1 ? (double)G : (double)((G + s - 1) / s) + meet);
        if (takes < least) {
            least = takes;
            c = s;
            plan.full = s == 1 ? tiles : rounds * ctas;
            grid = s == 1 ? std::min(tiles, ctas) : rounds > 0 ? ctas : rest * s;
        }
    }
    plan.split = c;
    const bool wide_y = aligned(a.y, 32) && a.ldy % 16 == 0, wide_h = aligned(a.hq, 32);
    if (c == 1)
        return launch_pdl(where, kern, dim3((unsigned)grid), dim3(kThreads), smem, stream, t0, t1, tx, a, plan, wide_y, wide_h, wait_limit,
                          stall);
    return launch_pdl_cluster(where, kern, dim3((unsigned)grid), dim3(kThreads), smem, stream, c, t0, t1, tx, a, plan, wide_y, wide_h, wait_limit,
                              stall);
}

}  // namespace f8t

}  // namespace

namespace f8b {

int launch_tile(const char *where, const uint8_t *xq, const uint8_t *w0, const uint8_t *w1, const Args &a, cudaStream_t stream,
                uint32_t wait_limit, int stall) {
    const bool apart = a.y != nullptr && (!aligned(a.y, 16) || a.ldy % 8 != 0);           // rows on no 16-byte boundary
    if (w1 != nullptr)
        return apart ? f8t::launch<true, true>(where, xq, w0, w1, a, stream, wait_limit, stall)
                     : f8t::launch<true, false>(where, xq, w0, w1, a, stream, wait_limit, stall);
    return apart ? f8t::launch<false, true>(where, xq, w0, w1, a, stream, wait_limit, stall)
                 : f8t::launch<false, false>(where, xq, w0, w1, a, stream, wait_limit, stall);
}

}  // namespace f8b

}  // namespace qspec
