// fp8_block_stream.cu -- products of E4M3 codes with a scale for each block of 128
// for few tokens: the linear, and the gate and up projections with SiLU,
// product and quantisation in one kernel.
//
//   y[m][n] = bf16(sum_g sa[g][m] sw[n / 128][g] sum_{k in g} xq[m][k] w8[n][k])
//   gated: h = silu(gate) up, out as E4M3 with a scale per token and 128 and / or bf16
//
// The weights are read once, so HBM bounds it: 128 output channels are the lanes
// of the accumulator, up to 128 tokens its columns (gated: up to 64, for each of the
// two parts).  TMA fills a ring of stages, one block of K to a stage (128 x 128 bytes of
// weights, twice for the gated one, and the tokens' 128 bytes each); one warp issues the
// products of a block into an accumulator of its own, and eight warps (thread = channel,
// half the tokens each) add it to their registers in fp32, times the block's scales, while
// the next blocks' products run.  The scales' products (token times weight) are made by
// a warp of its own, some blocks ahead.
// K is split over the CTAs of a cluster where the channels alone would leave
// multiprocessors idle; the parts meet in shared memory, in the order of K: a warp
// takes a token, its lanes four channels each, so that the maximum of 128 channels
// that a scale needs is a warp's.
// Measured: one token 4096 x 14336 in 11.7 us (5.0 TB/s), gated 14336 x 4096 in 20.2 us (5.8);
// 3 us of it are the way to the first block and from the last one, which a shorter call
// (4096 x 4096, 5.9 us) shows.  K in 4 / 8 parts: 12.9 / 11.8 us; gated in 1 / 2 / 4: 22.8 / 20.2 / 24.6.
#include <algorithm>

#include "fp8_block_host.h"
#include "umma.cuh"

namespace qspec {

namespace {

namespace f8s {

using f8b::Args;
using f8b::desc_sw128;
using f8b::f2;
using f8b::fma2;
using f8b::hi32;
using f8b::lo32;

constexpr int kTile = 128;                       // channels per CTA, and K per stage
constexpr int kWorkWarps = 8, kWork = 32 * kWorkWarps, kLoadWarp = 8, kMmaWarp = 9, kScaleWarp = 10, kThreads = kWork + 128;
constexpr int kBatch = 4, kBatches = 2;          // scales: blocks per hand-over, hand-overs in flight
using f8b::kMaxSplit;

// BN: most tokens (the products take bn of them, a multiple of 16)
template <int BN, bool kGated>
struct Cfg {
    static constexpr int kParts = kGated ? 2 : 1, kHalf = BN / 2;
    static constexpr int kCols = BN * kParts;                    // accumulator columns of one block
    static constexpr int kStage = kTile * kTile * kParts + BN * kTile;
    static constexpr int kOcc = kCols <= 64 && kStage <= 36 * 1024 - 1024 ? 2 : 1;    // CTAs per SM, as stages and sums allow
    static constexpr int kFit = 512 / kOcc / kCols < 4 ? 512 / kOcc / kCols : 4;      // accumulators in tensor memory
    static constexpr int kCtl = 512, kScales = kBatch * kBatches * kCols * 4;        // barriers; scales of blocks to come
    static constexpr int kBudget = (kOcc == 2 ? 112 : 224) * 1024 - 1024 - kCtl - kScales;
    static constexpr int kStages = kBudget / kStage < 8 ? kBudget / kStage : 8;
    // A stage's barrier also tells the work of its sums: it must not complete twice while a warp has yet to look at it, so
    // the products of the block that next uses the stage wait for all warps to have read this one's
    static constexpr int kBufs = kFit < kStages ? kFit : kStages;
    static constexpr uint32_t kAlloc = kBufs * kCols <= 32 ? 32 : kBufs * kCols <= 64 ? 64 : kBufs * kCols <= 128 ? 128 : kBufs * kCols <= 256 ? 256 : 512;
    static constexpr int kJoin = kCols * kTile * 4;              // a CTA's sums, over the stages
    static_assert(kStages >= 3 && kJoin <= kStages * kStage, "shared memory");
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kCtl + kScales;
    // registers per thread at launch and after the warps have shared them out
    static constexpr int kRegs = kOcc == 2 ? 80 : 168, kRegsWork = kOcc == 2 ? 96 : 200, kRegsRest = kOcc == 2 ? 48 : 96;
    static_assert(kOcc * kThreads * kRegs <= 65536 && kWork * kRegsWork + 128 * kRegsRest <= kThreads * kRegs, "register shares");
};

template <int BN, bool kGated>
__global__ void __launch_bounds__(kThreads, (Cfg<BN, kGated>::kOcc))
    stream_kernel(const __grid_constant__ CUtensorMap t0, const __grid_constant__ CUtensorMap t1,
                  const __grid_constant__ CUtensorMap tx, const __grid_constant__ Args a, int bn, int split, uint32_t wait_limit,
                  int stall) {
    using C = Cfg<BN, kGated>;
    constexpr int S = C::kStages, kParts = C::kParts, kHalf = C::kHalf, kLd = kHalf < 16 ? kHalf : 16;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stages = smem_raw + ((1024u - (umma::smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(stages + (size_t)S * C::kStage);
    uint64_t *done = full + S, *acc_empty = done + S, *scale_full = acc_empty + C::kBufs, *scale_empty = scale_full + kBatches,
             *drain = scale_empty + kBatches;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *timeout = reinterpret_cast<volatile int *>(tslot + 1);
    float *scales = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(full) + C::kCtl);     // [slot][part][token]
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x % (unsigned)split), tile = (int)(blockIdx.x / (unsigned)split);
    const int n0 = tile * kTile;
    const int G = a.K / kGroup;
    const int k0 = (int)((long long)G * rank / split), nk = (int)((long long)G * (rank + 1) / split) - k0;
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (umma::mbar_try_wait(bar, parity & 1)) return true;
        if (*timeout) return false;
        if (umma::mbar_wait(bar, parity & 1, wait_limit)) return true;
        *timeout = 1;
        return false;
    };
    auto all = [](bool mine) { return __all_sync(0xffffffffu, mine) != 0; };
    const uint32_t bytes = (uint32_t)(kParts * kTile * kTile + bn * kTile);
    auto load_weights = [&](int i) {
        uint8_t *stg = stages + (size_t)(i % S) * C::kStage;
        umma::mbar_arrive_expect_tx(&full[i % S], bytes);
        umma::tma_load_2d(stg, &t0, (k0 + i) * kGroup, n0, &full[i % S]);
        if (kGated) umma::tma_load_2d(stg + kTile * kTile, &t1, (k0 + i) * kGroup, n0, &full[i % S]);
    };
    auto load_tokens = [&](int i) {
        umma::tma_load_2d(stages + (size_t)(i % S) * C::kStage + kParts * kTile * kTile, &tx, (k0 + i) * kGroup, 0, &full[i % S]);
    };

    const bool elected = umma::elect_one();
    const int pre = min(S, nk);
    if (warp == kLoadWarp && elected) {
        *timeout = 0;
        for (int i = 0; i < S; ++i) {
            umma::mbar_init(&full[i], 1);
            umma::mbar_init(&done[i], 1);
        }
        for (int i = 0; i < C::kBufs; ++i) umma::mbar_init(&acc_empty[i], kWorkWarps);
        for (int i = 0; i < kBatches; ++i) {
            umma::mbar_init(&scale_full[i], 1);
            umma::mbar_init(&scale_empty[i], kWorkWarps);
        }
        umma::mbar_init(drain, 1);
        umma::mbar_fence_init();
        umma::fence_proxy_async();
        umma::fence_proxy_async_global();           // (the weights may be the kernel's in front, which is complete)
        // the first stages' weights at once, before the dependency wait too
        for (int i = 0; i < pre; ++i) load_weights(i);
    }
    if (warp == kMmaWarp) umma::tmem_alloc(tslot, C::kAlloc);
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    pdl_launch_dependents();
    const uint32_t tmem = *tslot;
    int loads = 0, issued = 0;
    // all warps' way to the end: the CTA's, then (behind a timeout's drain) the cluster's barrier
    auto meet = [&]() {
        if (split > 1)
            umma::cluster_sync();
        else
            __syncthreads();
    };

    if (warp >= kWorkWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kRegsRest));
        if (warp == kLoadWarp) {
            pdl_wait();
            if (elected)
                for (int i = 0; i < pre; ++i) load_tokens(i);
            __syncwarp();
            loads = pre;
            for (int i = pre; i < nk; ++i) {
                if (!all(wait(&done[i % S], (uint32_t)(i / S + 1)))) break;
                if (elected) {
                    load_weights(i);
                    load_tokens(i);
                }
                __syncwarp();
                loads = i + 1;
            }
        } else if (warp == kMmaWarp) {
            const uint32_t idesc = umma::instr_desc(0, 0, kTile, bn);            // e4m3 x e4m3 -> f32
            pdl_wait();
            const bool go = !stall || all(wait(drain, 0));       // (tests: nothing arrives there before the end)
            for (int i = 0; go && i < nk; ++i) {
                const int s = i % S, b = i % C::kBufs;
                if (!all(wait(&full[s], (uint32_t)(i / S))) || !all(wait(&acc_empty[b], (uint32_t)(i / C::kBufs + 1)))) break;
                umma::fence_after_sync();
                const uint32_t at = umma::smem_addr(stages + (size_t)s * C::kStage);
                const uint64_t bd = desc_sw128(at + kParts * kTile * kTile);
                if (elected) {
#pragma unroll
                    for (int p = 0; p < kParts; ++p) {
                        const uint64_t ad = desc_sw128(at + p * kTile * kTile);
#pragma unroll
                        for (int kk = 0; kk < kGroup / 32; ++kk)                 // K = 32 bytes per MMA: +2 in the address field
                            umma::mma_e4m3(tmem + b * C::kCols + p * BN, ad + 2 * kk, bd + 2 * kk, idesc, kk != 0 ? 1u : 0u);
                    }
                    umma::mma_commit(&done[s]);                                  // the stage is free, the sums are there
                }
                __syncwarp();
                issued = i + 1;
            }
        } else if (warp == kScaleWarp) {
            constexpr int kEach = (BN + 31) / 32;
            const float *w0 = a.s0 + (size_t)tile * G + k0, *w1 = kGated ? a.s1 + (size_t)tile * G + k0 : nullptr;
            // (coherent loads, past L1: the kernel in front may write either kind of scales while this one is resident, and
            // a product before it may have left their old values in this multiprocessor's L1)
            pdl_wait();
            for (int base = 0; base < nk; base += kBatch) {
                float x[kBatch][kEach], s0[kBatch], s1[kBatch];
#pragma unroll
                for (int u = 0; u < kBatch; ++u) {
                    const bool some = base + u < nk;
                    s0[u] = some ? __ldcg(w0 + base + u) : 0.0f;
                    s1[u] = some && kGated ? __ldcg(w1 + base + u) : 0.0f;
#pragma unroll
                    for (int e = 0; e < kEach; ++e) {
                        const int m = lane + 32 * e;
                        x[u][e] = some && m < a.M ? __ldcg(a.sa + (size_t)(k0 + base + u) * a.lds + m) : 0.0f;
                    }
                }
                const int slot = base / kBatch % kBatches;
                if (!all(wait(&scale_empty[slot], (uint32_t)(base / (kBatch * kBatches) + 1)))) break;
#pragma unroll
                for (int u = 0; u < kBatch; ++u)
#pragma unroll
                    for (int e = 0; e < kEach; ++e)
                        if (BN >= 32 || lane < BN) {
                            float *at = scales + (slot * kBatch + u) * C::kCols + lane + 32 * e;
                            at[0] = x[u][e] * s0[u];
                            if (kGated) at[BN] = x[u][e] * s1[u];
                        }
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&scale_full[slot]);
            }
        }
        // after a timeout: the copies and products in flight finish (bounded) before the memory they use is used
        // again; both issuers stopped at the timeout, so at most S copies are outstanding
        __syncthreads();
        if (*timeout) {
            if (warp == kLoadWarp && elected)
                for (int b = max(0, loads - S); b < loads; ++b) umma::mbar_wait(&full[b % S], (uint32_t)((b / S) & 1), kWaitLimit);
            if (warp == kMmaWarp && elected && issued > 0) {
                umma::mma_commit(drain);
                umma::mbar_wait(drain, 0, kWaitLimit);
            }
            if (warp == kScaleWarp && lane == 0) flag(a.st, QSPEC_ERR_TIMEOUT);
            __syncwarp();
        }
        // (freed before the cluster's barrier: a CTA that waits for its peers holds no tensor memory that one of them may
        // be waiting for, behind another stream's kernel)
        umma::fence_after_sync();
        if (warp == kMmaWarp) umma::tmem_free(tmem, C::kAlloc);
        meet();
    } else {
        asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kRegsWork));
        // ---- thread = channel, half the tokens: sum over the blocks ----
        const int half = bn / 2, c0 = (warp >> 2) * half;        // its tokens: c0 .. c0 + half - 1
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        uint64_t acc[kParts][kHalf / 2];
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int j = 0; j < kHalf / 2; ++j) acc[p][j] = 0;
        bool ok = true;
        pdl_wait();
        for (int i = 0; i < nk; ++i) {
            const int b = i % C::kBufs, at = i % (kBatch * kBatches), slot = at / kBatch;
            if (at % kBatch == 0 && !(ok = all(wait(&scale_full[slot], (uint32_t)(i / (kBatch * kBatches)))))) break;
            if (!(ok = all(wait(&done[i % S], (uint32_t)(i / S))))) break;
            umma::fence_after_sync();
            const float *sc = scales + at * C::kCols + c0;
            const uint32_t from = tmem + lanes + b * C::kCols + c0;
            // a chunk is on its way while the one before it is added (the last ones may reach past the half's tokens:
            // into columns of the accumulator whose sums nobody looks at)
            constexpr int kChunks = kHalf / kLd, kAll = kParts * kChunks;
            uint32_t d[2][kLd];
            umma::tmem_ld_cols<kLd>(from, d[0]);
#pragma unroll
            for (int c = 0; c < kAll; ++c) {
                const int p = c / kChunks, j0 = c % kChunks * kLd;
                umma::tmem_ld_wait();
                if (c + 1 < kAll) {
                    const int p1 = (c + 1) / kChunks, j1 = (c + 1) % kChunks * kLd;
                    if (j1 < half) umma::tmem_ld_cols<kLd>(from + p1 * BN + j1, d[(c + 1) & 1]);
                } else {
                    umma::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) umma::mbar_arrive(&acc_empty[b]);
                }
                if (j0 < half) {
#pragma unroll
                    for (int j = 0; j < kLd; j += 4) {
                        const ulonglong2 f = *reinterpret_cast<const ulonglong2 *>(sc + p * BN + j0 + j);
                        acc[p][(j0 + j) / 2] = fma2(f2(__uint_as_float(d[c & 1][j]), __uint_as_float(d[c & 1][j + 1])), f.x, acc[p][(j0 + j) / 2]);
                        acc[p][(j0 + j) / 2 + 1] =
                            fma2(f2(__uint_as_float(d[c & 1][j + 2]), __uint_as_float(d[c & 1][j + 3])), f.y, acc[p][(j0 + j) / 2 + 1]);
                    }
                }
            }
            if (at % kBatch == kBatch - 1) {
                __syncwarp();
                if (lane == 0) umma::mbar_arrive(&scale_empty[slot]);
            }
        }
        // ---- the parts of K meet: [part][token][channel] over the stages, whose last products are done ----
        const int tokens = a.M;
        float *sums = reinterpret_cast<float *>(stages);
        if (ok) {
            const int ch = 32 * (warp & 3) + lane;
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
                for (int j = 0; j < kHalf; j += 2) {
                    if (j < half && c0 + j < tokens) sums[(p * BN + c0 + j) * kTile + ch] = lo32(acc[p][j / 2]);
                    if (j + 1 < half && c0 + j + 1 < tokens) sums[(p * BN + c0 + j + 1) * kTile + ch] = hi32(acc[p][j / 2]);
                }
        }
        __syncthreads();
        meet();
        const int n = n0 + 4 * lane;
        for (int c = warp * split + rank; c < tokens; c += kWorkWarps * split) {
            float v[kParts][4];
            const float *at[kParts];
#pragma unroll
            for (int p = 0; p < kParts; ++p) at[p] = sums + (p * BN + c) * kTile + 4 * lane;
            if (split > 1) {
                f8b::sum_parts(at, split, 0, v);
            } else {
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    const float4 f = *reinterpret_cast<const float4 *>(at[p]);
                    v[p][0] = f.x, v[p][1] = f.y, v[p][2] = f.z, v[p][3] = f.w;
                }
            }
            if constexpr (kGated)
                f8b::store_gated(a, c, tile, lane, v[0], v[1]);
            else
                f8b::store_bf16(a, c, n, v[0]);
        }
    }
    if (split > 1) umma::cluster_sync();         // (a peer may still read this CTA's sums)
}

template <int BN, bool kGated>
struct Kernel {
    static const void *address() { return reinterpret_cast<const void *>(stream_kernel<BN, kGated>); }
    static constexpr int threads = kThreads, per = Cfg<BN, kGated>::kOcc;
    static constexpr size_t smem = Cfg<BN, kGated>::kSmem;
    static constexpr bool carveout = true;
};
template <int BN, bool kGated>
int slots() { return sm_count() * Cfg<BN, kGated>::kOcc; }       // CTAs that run at once
// The same in clusters of s.  Where two CTAs share an SM the runtime's count takes one for what fits: there a twentieth is left
// free for what clusters of four or more cannot fill, 288 of 304 CTAs.  (Clusters of eight: 264, 272, 280 and 288 CTAs run at
// once, 296 do not: 1 x N x 4096 with 33 / 34 / 35 / 36 / 37 tiles 6.0 / 6.1 / 6.3 / 6.7 / 9.8 us in eight parts, 6.0 / 6.1 / 6.2 / 6.3 /
// 6.3 in six; K = 14336 12.1 / 12.6 / 12.7 / 13.3 / 17.8 and 12.7 / 12.9 / 13.1 / 13.3 / 13.6.  1 x 9600 x 4096, 75 tiles, in four 12.3, in
// three 8.8.)
template <int BN, bool kGated>
int room(int s) {
    if (Cfg<BN, kGated>::kOcc == 1) return f8b::resident<Kernel<BN, kGated>>().ctas[s];
    return s >= 4 ? slots<BN, kGated>() * 19 / 20 : slots<BN, kGated>();
}

// Parts of K: doubled as long as there is room and two blocks for each; then three, five or six where they shorten the
// longest part by a fifth and leave a tenth of the machine free, which the clusters of such sizes cannot all fill (us, with
// powers of two / best: 1 x 5120 x 13824, 40 tiles, four 14.5 / six 13.7, seven do not fit 18.9; 128 x 5120 x 13824 two 27.6 /
// three 21.2; 1 x 10240 x 8192 two 16.6 / three 15.5; but 1 x 6144 x 4096 four 6.6 / five 7.1, 80 x 3584 x 3584, 28 tiles, four 7.6 /
// five 9.2.)
template <int BN, bool kGated>
int parts(int tiles, int G) {
    const long long all = slots<BN, kGated>();
    int split = 1;
    while (split < kMaxSplit && (long long)tiles * split * 2 <= room<BN, kGated>(split * 2) && G / (split * 2) >= 2) split *= 2;
    for (int s : {3, 5, 6})
        if (s > split && (long long)tiles * s * 10 <= all * 9 && tiles * s <= room<BN, kGated>(s) && G / s >= 2 && (G + s - 1) / s * 5 <= (G + split - 1) / split * 4) split = s;
    return split;
}

template <int BN, bool kGated>
int launch(const char *where, const uint8_t *xq, const uint8_t *w0, const uint8_t *w1, const Args &a, int bn,
           cudaStream_t stream, uint32_t wait_limit, int stall) {
    using C = Cfg<BN, kGated>;
    CUtensorMap t0, t1, tx;
    if (byte_tmap_sw128(&t0, w0, a.N, a.K, (size_t)a.K, kTile) ||
        (kGated && byte_tmap_sw128(&t1, w1, a.N, a.K, (size_t)a.K, kTile)) ||
        byte_tmap_sw128(&tx, xq, a.M, a.K, (size_t)a.K, bn))
        return QSPEC_ERR_UNSUPPORTED;
    if (!kGated) t1 = t0;
    auto kern = stream_kernel<BN, kGated>;
    int rc = smem_limit_once(reinterpret_cast<const void *>(kern), (int)C::kSmem, true);
    if (rc) return rc;
    const int tiles = (a.N + kTile - 1) / kTile;
    const int split = parts<BN, kGated>(tiles, a.K / kGroup);
    if (split == 1)
        return launch_pdl(where, kern, dim3((unsigned)tiles), dim3(kThreads), C::kSmem, stream, t0, t1, tx, a, bn, split, wait_limit, stall);
    return launch_pdl_cluster(where, kern, dim3((unsigned)(tiles * split)), dim3(kThreads), C::kSmem, stream, split, t0, t1, tx, a, bn, split, wait_limit, stall);
}

// Few tokens here, many in tiles of 128 (fp8_block_tile.cu): 128 channels by M tokens against 128 tokens by 256 channels.
// Up to 16 tokens here.  Up to 32 (gated), 64 and 128 here too while the channels' tiles fit the machine at once, since a CTA
// goes through one tile, and up to 64 behind the gate while they fit it twice; above 64 tokens not where a CTA has 48 blocks of K or more, above 96 not from 32, which take longer
// than the many-token kernel's.  Measured here / there, us: 72 x 28672 x 8192 52.9 / 41.4, 48 x 128256 x 4096 91.9 / 85.1, 64 x 28672 x 4096 22.9 / 23.4, 80
// x 4096 x 4096 8.4 / 10.4, 96 x 14336 x 4096 15.8 / 16.2, 96 x 10240 x 8192 (64 blocks) 25.8 / 20.8, 128 x 14336 x 4096 (32) 18.1 / 16.8, 128 x 4096 x 14336 (28) 17.5 /
// 19.0; gated 32 x 14336 x 4096 21.6 / 22.8, 32 x 24576 x 4096 41.3 / 37.4, 16 x 28672 x 8192 70.9 / 74.7, 48 x 4096 x 4096 10.7 / 11.9, 48 x 9216 x
// 4096 17.1 / 18.3, 48 x 11008 x 4096 20.9 / 20.5.
template <bool kGated>
int launch_any(const char *where, const uint8_t *xq, const uint8_t *w0, const uint8_t *w1, const Args &a, cudaStream_t st,
               uint32_t wait_limit = kWaitLimit, int stall = 0) {
    const int bn = (a.M + 15) / 16 * 16, tiles = (a.N + kTile - 1) / kTile, G = a.K / kGroup;
    if (bn <= 16) return launch<16, kGated>(where, xq, w0, w1, a, bn, st, wait_limit, stall);
    if (bn <= 32 && (!kGated || tiles <= slots<32, kGated>())) return launch<32, kGated>(where, xq, w0, w1, a, bn, st, wait_limit, stall);
    if constexpr (kGated) {
        if (bn > 32 && bn <= 64 && tiles * 2LL <= slots<64, kGated>()) return launch<64, kGated>(where, xq, w0, w1, a, bn, st, wait_limit, stall);
    } else {
        if (bn <= 64 && tiles <= slots<64, kGated>()) return launch<64, kGated>(where, xq, w0, w1, a, bn, st, wait_limit, stall);
        if (bn > 64 && bn <= 128 && tiles <= slots<128, kGated>()) {
            const int p = parts<128, kGated>(tiles, G);
            if ((G + p - 1) / p < (bn <= 96 ? 48 : 32)) return launch<128, kGated>(where, xq, w0, w1, a, bn, st, wait_limit, stall);
        }
    }
    return f8b::launch_tile(where, xq, w0, w1, a, st, wait_limit, stall);
}

}  // namespace f8s

}  // namespace

}  // namespace qspec

using namespace qspec;

namespace {

int check_linear(const uint8_t *xq, const float *sa, int lds, const uint8_t *w8, const float *sw, int M, int N, int K,
                 const uint16_t *y_bf16, int ldy) {
    if (!xq || !sa || !w8 || !sw || !y_bf16) return QSPEC_ERR_NULL;
    if (M < 1 || M > f8b::kMaxM || N < 1 || N > f8b::kMaxN || K < kGroup || K % kGroup || ldy < N || lds < M)
        return QSPEC_ERR_SHAPE;
    if (!aligned(xq, 16) || !aligned(w8, 16) || !aligned(sa, 4) || !aligned(sw, 4) || !aligned(y_bf16, 2))
        return QSPEC_ERR_ALIGN;
    return check_device();
}

int check_gated(const uint8_t *xq, const float *sa, int lds, const uint8_t *w_gate, const float *s_gate, const uint8_t *w_up,
                const float *s_up, int M, int N, int K, const uint8_t *hq, const float *sh, int ldh, const uint16_t *h_bf16,
                int ldy) {
    if (!xq || !sa || !w_gate || !s_gate || !w_up || !s_up || (hq != nullptr) != (sh != nullptr) || (!hq && !h_bf16))
        return QSPEC_ERR_NULL;
    if (M < 1 || M > f8b::kMaxM || N < kGroup || N > f8b::kMaxN || N % kGroup || K < kGroup || K % kGroup || lds < M ||
        (hq && ldh < M) || (h_bf16 && ldy < N))
        return QSPEC_ERR_SHAPE;
    if (!aligned(xq, 16) || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(sa, 4) || !aligned(s_gate, 4) ||
        !aligned(s_up, 4) || (hq && (!aligned(hq, 16) || !aligned(sh, 4))) || (h_bf16 && !aligned(h_bf16, 2)))
        return QSPEC_ERR_ALIGN;
    return check_device();
}

}  // namespace

extern "C" int qspec_linear_fp8_block(const uint8_t *xq, const float *sa, int lds, const uint8_t *w8, const float *sw, int M,
                                      int N, int K, uint16_t *y_bf16, int ldy, int32_t *dev_status, qspec_stream_t stream) {
    const int rc = check_linear(xq, sa, lds, w8, sw, M, N, K, y_bf16, ldy);
    if (rc) return rc;
    const f8b::Args a = {sa, sw, nullptr, y_bf16, nullptr, nullptr, dev_status, lds, M, N, K, ldy, 0};
    return f8s::launch_any<false>("qspec_linear_fp8_block", xq, w8, nullptr, a, as_cuda(stream));
}

extern "C" int qspec_gated_fp8_block(const uint8_t *xq, const float *sa, int lds, const uint8_t *w_gate, const float *s_gate,
                                     const uint8_t *w_up, const float *s_up, int M, int N, int K, uint8_t *hq, float *sh,
                                     int ldh, uint16_t *h_bf16, int ldy, int32_t *dev_status, qspec_stream_t stream) {
    const int rc = check_gated(xq, sa, lds, w_gate, s_gate, w_up, s_up, M, N, K, hq, sh, ldh, h_bf16, ldy);
    if (rc) return rc;
    const f8b::Args a = {sa, s_gate, s_up, h_bf16, hq, sh, dev_status, lds, M, N, K, ldy, ldh};
    return f8s::launch_any<true>("qspec_gated_fp8_block", xq, w_gate, w_up, a, as_cuda(stream));
}

extern "C" int qspec_debug_fp8_block_bounded(const uint8_t *xq, const float *sa, int lds, const uint8_t *w0, const float *s0,
                                             const uint8_t *w1, const float *s1, int M, int N, int K, uint8_t *hq, float *sh,
                                             int ldh, uint16_t *y_bf16, int ldy, uint32_t wait_limit, int stall,
                                             int32_t *dev_status, qspec_stream_t stream) {
    if (wait_limit < 1) return QSPEC_ERR_SHAPE;
    const bool gated = w1 != nullptr;
    const int rc = gated ? check_gated(xq, sa, lds, w0, s0, w1, s1, M, N, K, hq, sh, ldh, y_bf16, ldy)
                         : check_linear(xq, sa, lds, w0, s0, M, N, K, y_bf16, ldy);
    if (rc) return rc;
    const f8b::Args a = {sa, s0, s1, y_bf16, hq, sh, dev_status, lds, M, N, K, ldy, ldh};
    return gated ? f8s::launch_any<true>("qspec_debug_fp8_block_bounded", xq, w0, w1, a, as_cuda(stream), wait_limit, stall)
                 : f8s::launch_any<false>("qspec_debug_fp8_block_bounded", xq, w0, nullptr, a, as_cuda(stream), wait_limit, stall);
}
