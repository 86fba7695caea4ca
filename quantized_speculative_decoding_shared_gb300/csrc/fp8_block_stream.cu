// fp8_block_stream.cu -- products of E4M3 codes with a scale for each block of 128
// for few tokens: the linear, and the gate and up projections with SiLU,
// product and quantisation in one kernel.
//
//   y[m][n] = bf16(sum_g sa[g][m] sw[n / 128][g] sum_{k in g} xq[m][k] w8[n][k])
//   gated: h = silu(gate) up, out as E4M3 with a scale per token and 128 and / or bf16
//
// The weights are read once, so HBM bounds it: 128 output channels are the lanes
// of the accumulator, BN tokens its columns.  TMA fills a ring of stages, one
// block of K to a stage (128 x 128 bytes of weights, twice for the gated one, and
// BN x 128 of the tokens); one lane issues the four products of a block into an
// accumulator of its own, and eight warps (thread = channel, half the tokens each)
// add it to their registers in fp32, times the block's two scales, while the next
// block's products run.
// K is split over the CTAs of a cluster where the channels alone would leave
// multiprocessors idle; the parts meet in shared memory, in the order of K: a warp
// takes a token, its lanes four channels each, so that the maximum of 128 channels
// that a scale needs is a warp's.
#include <algorithm>

#include "fp8_block_host.h"
#include "umma.cuh"

namespace qspec {

namespace {

namespace f8s {

using f8b::Args;

constexpr int kTile = 128;                       // channels per CTA, and K per stage
constexpr int kWorkWarps = 8, kLoadWarp = 8, kMmaWarp = 9, kThreads = 320;

template <int BN, bool kGated>
struct Cfg {
    static constexpr int kParts = kGated ? 2 : 1;
    static constexpr int kCols = BN * kParts;                    // accumulator columns of one block
    static constexpr int kStage = kTile * kTile * kParts + BN * kTile;
    static constexpr int kOcc = BN / 2 * kParts <= 64 ? 2 : 1;   // CTAs per SM: as the sums leave registers for
    static constexpr int kTmem = kOcc == 2 ? 256 : 512;
    static constexpr int kBufs = kTmem / kCols < 4 ? kTmem / kCols : 4;
    static constexpr uint32_t kAlloc = kBufs * kCols < 32 ? 32 : kBufs * kCols;
    static constexpr int kBudget = kOcc == 2 ? 110 * 1024 : 220 * 1024;
    static constexpr int kCtl = 1024 + 2 * kWorkWarps * (BN / 2) * 4 * kParts;        // barriers; scales of the warps
    static constexpr int kStages = (kBudget - 1024 - kCtl) / kStage < 8 ? (kBudget - 1024 - kCtl) / kStage : 8;
    static constexpr int kJoin = kCols * kTile * 4;              // a CTA's sums, over the stages
    static_assert(kStages >= 2 && kJoin <= kStages * kStage, "shared memory");
    static constexpr size_t kSmem = 1024 + (size_t)kStages * kStage + kCtl;
};

__device__ __forceinline__ uint64_t desc_sw128(uint32_t saddr) {       // K-major, rows of 128 bytes, 128-byte swizzle
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 | (uint64_t)1 << 46 |
           (uint64_t)2 << 61;
}

template <int BN, bool kGated>
__global__ void __launch_bounds__(kThreads, (Cfg<BN, kGated>::kOcc))
    stream_kernel(const __grid_constant__ CUtensorMap t0, const __grid_constant__ CUtensorMap t1,
                  const __grid_constant__ CUtensorMap tx, const __grid_constant__ Args a, int split, uint32_t wait_limit) {
    using C = Cfg<BN, kGated>;
    constexpr int S = C::kStages, kParts = C::kParts, kHalf = BN / 2, kLd = kHalf < 16 ? kHalf : 16;   // (32 at a time spill)
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *stages = smem_raw + ((1024u - (umma::smem_addr(smem_raw) & 1023u)) & 1023u);
    uint64_t *full = reinterpret_cast<uint64_t *>(stages + (size_t)S * C::kStage);
    uint64_t *empty = full + S, *acc_full = empty + S, *acc_empty = acc_full + C::kBufs, *drain = acc_empty + C::kBufs;
    uint32_t *tslot = reinterpret_cast<uint32_t *>(drain + 1);
    volatile int *timeout = reinterpret_cast<volatile int *>(tslot + 1);
    float *scales = reinterpret_cast<float *>(reinterpret_cast<uint8_t *>(full) + 1024);
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int rank = (int)(blockIdx.x % (unsigned)split), tile = (int)(blockIdx.x / (unsigned)split);
    const int n0 = tile * kTile, m0 = blockIdx.y * BN;
    const int G = a.K / kGroup;
    const int k0 = (int)((long long)G * rank / split), k1 = (int)((long long)G * (rank + 1) / split), nk = k1 - k0;
    auto wait = [&](uint64_t *bar, uint32_t parity) -> bool {
        if (*timeout) return false;
        if (umma::mbar_wait(bar, parity & 1, wait_limit)) return true;
        *timeout = 1;
        return false;
    };

    if (threadIdx.x == 0) {
        *timeout = 0;
        for (int i = 0; i < S; ++i) {
            umma::mbar_init(&full[i], 1);
            umma::mbar_init(&empty[i], 1);
        }
        for (int i = 0; i < C::kBufs; ++i) {
            umma::mbar_init(&acc_full[i], 1);
            umma::mbar_init(&acc_empty[i], kWorkWarps);
        }
        umma::mbar_init(drain, 1);
        umma::mbar_fence_init();
    }
    if (warp == kMmaWarp) umma::tmem_alloc(tslot, C::kAlloc);
    if (warp == kLoadWarp && lane == 0) {
        umma::prefetch_tmap(&t0);
        if (kGated) umma::prefetch_tmap(&t1);
        umma::prefetch_tmap(&tx);
    }
    umma::fence_before_sync();
    __syncthreads();
    umma::fence_after_sync();
    pdl_launch_dependents();
    const uint32_t tmem = *tslot;
    int loads = 0, issued = 0;
    float acc[kParts][kHalf];

    if (warp == kLoadWarp) {
        if (lane == 0) {
            auto weights = [&](int i) {
                uint8_t *stg = stages + (size_t)(i % S) * C::kStage;
                umma::mbar_arrive_expect_tx(&full[i % S], C::kStage);
                umma::tma_load_2d(stg, &t0, (k0 + i) * kGroup, n0, &full[i % S]);
                if (kGated) umma::tma_load_2d(stg + kTile * kTile, &t1, (k0 + i) * kGroup, n0, &full[i % S]);
            };
            auto tokens = [&](int i) {
                umma::tma_load_2d(stages + (size_t)(i % S) * C::kStage + kParts * kTile * kTile, &tx, (k0 + i) * kGroup, m0,
                                  &full[i % S]);
            };
            // the first stages' weights before the dependency wait (they are immutable)
            const int pre = min(S, nk);
            for (int i = 0; i < pre; ++i) weights(i);
            pdl_wait();
            for (int i = 0; i < pre; ++i) tokens(i);
            loads = pre;
            for (int i = pre; i < nk; ++i) {
                if (!wait(&empty[i % S], (uint32_t)(i / S + 1))) break;
                weights(i);
                tokens(i);
                loads = i + 1;
            }
        }
    } else if (warp == kMmaWarp) {
        if (lane == 0) {
            constexpr uint32_t idesc = umma::instr_desc(0, 0, kTile, BN);        // e4m3 x e4m3 -> f32
            for (int i = 0; i < nk; ++i) {
                const int s = i % S, b = i % C::kBufs;
                if (!wait(&full[s], (uint32_t)(i / S)) || !wait(&acc_empty[b], (uint32_t)(i / C::kBufs + 1))) break;
                umma::fence_after_sync();
                const uint32_t at = umma::smem_addr(stages + (size_t)s * C::kStage);
                const uint64_t bd = desc_sw128(at + kParts * kTile * kTile);
#pragma unroll
                for (int p = 0; p < kParts; ++p) {
                    const uint64_t ad = desc_sw128(at + p * kTile * kTile);
#pragma unroll
                    for (int kk = 0; kk < kGroup / 32; ++kk)                     // K = 32 bytes per MMA: +2 in the address field
                        umma::mma_e4m3(tmem + b * C::kCols + p * BN, ad + 2 * kk, bd + 2 * kk, idesc, kk != 0 ? 1u : 0u);
                }
                umma::mma_commit(&empty[s]);
                umma::mma_commit(&acc_full[b]);
                issued = i + 1;
            }
        }
    } else {
        // ---- thread = channel, kHalf tokens: sum over the blocks ----
        const int c0 = (warp >> 2) * kHalf;                      // first of its tokens
        const uint32_t lanes = (uint32_t)(32 * (warp & 3)) << 16;
        float *mine = scales + warp * (2 * kHalf * kParts);      // its scales, two blocks' in turn
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int j = 0; j < kHalf; ++j) acc[p][j] = 0.0f;
        const float *w0 = a.s0 + (size_t)tile * G + k0, *w1 = kGated ? a.s1 + (size_t)tile * G + k0 : nullptr;
        constexpr int kEach = (kHalf + 31) / 32;
        float next[kEach], n0s = 0.0f, n1s = 0.0f;
        auto ask = [&](int i) {                                   // scales of block i
            n0s = __ldg(w0 + i);
            if (kGated) n1s = __ldg(w1 + i);
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int j = lane + 32 * e, m = m0 + c0 + j;
                next[e] = j < kHalf && m < a.M ? __ldg(a.sa + (size_t)(k0 + i) * a.lds + m) : 0.0f;
            }
        };
        pdl_wait();
        if (nk > 0) ask(0);
        for (int i = 0; i < nk; ++i) {
            const int b = i % C::kBufs;
            float *at = mine + (i & 1) * kHalf * kParts;
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                if (lane + 32 * e < kHalf) {
                    at[lane + 32 * e] = next[e] * n0s;
                    if (kGated) at[kHalf + lane + 32 * e] = next[e] * n1s;
                }
            if (i + 1 < nk) ask(i + 1);
            __syncwarp();
            if (!__all_sync(0xffffffffu, wait(&acc_full[b], (uint32_t)(i / C::kBufs)))) break;
            umma::fence_after_sync();
#pragma unroll
            for (int p = 0; p < kParts; ++p)
#pragma unroll
                for (int j0 = 0; j0 < kHalf; j0 += kLd) {
                    uint32_t d[kLd];
                    umma::tmem_ld_cols<kLd>(tmem + lanes + b * C::kCols + p * BN + c0 + j0, d);
                    umma::tmem_ld_wait();
#pragma unroll
                    for (int j = 0; j < kLd; j += 4) {
                        const float4 s = *reinterpret_cast<const float4 *>(at + p * kHalf + j0 + j);
                        acc[p][j0 + j] = fmaf(__uint_as_float(d[j]), s.x, acc[p][j0 + j]);
                        acc[p][j0 + j + 1] = fmaf(__uint_as_float(d[j + 1]), s.y, acc[p][j0 + j + 1]);
                        acc[p][j0 + j + 2] = fmaf(__uint_as_float(d[j + 2]), s.z, acc[p][j0 + j + 2]);
                        acc[p][j0 + j + 3] = fmaf(__uint_as_float(d[j + 3]), s.w, acc[p][j0 + j + 3]);
                    }
                }
            umma::fence_before_sync();
            __syncwarp();
            if (lane == 0) umma::mbar_arrive(&acc_empty[b]);
        }
    }

    // after a timeout: the copies and products in flight finish (bounded) before the memory they use is used
    // again; both issuers stopped at the timeout, so at most S copies are outstanding
    __syncthreads();
    if (*timeout) {
        if (warp == kLoadWarp && lane == 0)
            for (int b = max(0, loads - S); b < loads; ++b) umma::mbar_wait(&full[b % S], (uint32_t)((b / S) & 1), kWaitLimit);
        if (warp == kMmaWarp && lane == 0 && issued > 0) {
            umma::mma_commit(drain);
            umma::mbar_wait(drain, 0, kWaitLimit);
        }
        if (threadIdx.x == 0) flag(a.st, QSPEC_ERR_TIMEOUT);
    }
    umma::fence_before_sync();
    __syncthreads();
    if (warp == kMmaWarp) umma::tmem_free(tmem, C::kAlloc);

    // ---- the parts of K meet: [part][token][channel] over the stages ----
    float *sums = reinterpret_cast<float *>(stages);
    if (warp < kWorkWarps) {
        const int c0 = (warp >> 2) * kHalf, ch = 32 * (warp & 3) + lane;
#pragma unroll
        for (int p = 0; p < kParts; ++p)
#pragma unroll
            for (int j = 0; j < kHalf; ++j) sums[(p * BN + c0 + j) * kTile + ch] = acc[p][j];
    }
    if (split > 1)
        umma::cluster_sync();
    else
        __syncthreads();
    const int tokens = min(BN, a.M - m0);
    if (warp < kWorkWarps) {
        const int n = n0 + 4 * lane;
        for (int c = warp * split + rank; c < tokens; c += kWorkWarps * split) {
            const int m = m0 + c;
            float v[kParts][4];
#pragma unroll
            for (int p = 0; p < kParts; ++p) {
                const float *at = sums + (p * BN + c) * kTile + 4 * lane;
#pragma unroll
                for (int e = 0; e < 4; ++e) v[p][e] = 0.0f;
                for (int r = 0; r < split; ++r) {
                    float4 f;
                    if (split > 1) {
                        const uint4 w = umma::ld_peer_v4(at, (uint32_t)r);
                        f = make_float4(__uint_as_float(w.x), __uint_as_float(w.y), __uint_as_float(w.z), __uint_as_float(w.w));
                    } else {
                        f = *reinterpret_cast<const float4 *>(at);
                    }
                    v[p][0] += f.x;
                    v[p][1] += f.y;
                    v[p][2] += f.z;
                    v[p][3] += f.w;
                }
            }
            if constexpr (kGated) {
                float amax = 0.0f;
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    v[0][e] = f8b::gated(v[0][e], v[kParts - 1][e]);
                    asm("max.NaN.f32 %0, %0, %1;" : "+f"(amax) : "f"(fabsf(v[0][e])));
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) {
                    const float other = __shfl_xor_sync(0xffffffffu, amax, o);
                    asm("max.NaN.f32 %0, %0, %1;" : "+f"(amax) : "f"(other));
                }
                if (a.hq != nullptr) {
                    const f8b::Quant q(amax);
                    reinterpret_cast<uint32_t *>(a.hq + (size_t)m * a.N + n0)[lane] =
                        q.s == 0.0f ? 0u : f8b::codes4(v[0][0] * q.up * q.inv, v[0][1] * q.up * q.inv, v[0][2] * q.up * q.inv, v[0][3] * q.up * q.inv);
                    if (lane == 0) a.sh[(size_t)tile * a.ldh + m] = q.s;
                }
                if (lane == 0 && !(amax < (a.y != nullptr ? 3.3961775292304601e38f : INFINITY))) flag(a.st, QSPEC_ERR_NONFINITE);
            }
            if (!kGated || a.y != nullptr) {
                uint16_t *y = a.y + (size_t)m * a.ldy + n;
                if ((reinterpret_cast<uintptr_t>(y) & 7) == 0 && n + 4 <= a.N) {
                    *reinterpret_cast<uint2 *>(y) =
                        make_uint2((uint32_t)float_to_bf16_bits(v[0][0]) | (uint32_t)float_to_bf16_bits(v[0][1]) << 16,
                                   (uint32_t)float_to_bf16_bits(v[0][2]) | (uint32_t)float_to_bf16_bits(v[0][3]) << 16);
                } else {
#pragma unroll
                    for (int e = 0; e < 4; ++e)
                        if (n + e < a.N) y[e] = float_to_bf16_bits(v[0][e]);
                }
            }
        }
    }
    if (split > 1) umma::cluster_sync();         // (a peer may still read this CTA's sums)
}

template <int BN, bool kGated>
int launch(const char *where, const uint8_t *xq, const uint8_t *w0, const uint8_t *w1, const Args &a, cudaStream_t stream,
           uint32_t wait_limit) {
    using C = Cfg<BN, kGated>;
    CUtensorMap t0, t1, tx;
    if (byte_tmap_sw128(&t0, w0, a.N, a.K, (size_t)a.K, kTile) ||
        (kGated && byte_tmap_sw128(&t1, w1, a.N, a.K, (size_t)a.K, kTile)) ||
        byte_tmap_sw128(&tx, xq, a.M, a.K, (size_t)a.K, BN))
        return QSPEC_ERR_UNSUPPORTED;
    if (!kGated) t1 = t0;
    auto kern = stream_kernel<BN, kGated>;
    int rc = smem_limit_once(reinterpret_cast<const void *>(kern), (int)C::kSmem, true);
    if (rc) return rc;
    const int tiles = (a.N + kTile - 1) / kTile, rows = (a.M + BN - 1) / BN, G = a.K / kGroup;
    int split = 1;
    while (split < 8 && (long long)tiles * rows * split * 2 <= (long long)sm_count() * C::kOcc && G / (split * 2) >= 2) split *= 2;
    const dim3 grid((unsigned)(tiles * split), (unsigned)rows);
    if (split == 1)
        return launch_pdl(where, kern, grid, dim3(kThreads), C::kSmem, stream, t0, t1, tx, a, split, wait_limit);
    return launch_pdl_cluster(where, kern, grid, dim3(kThreads), C::kSmem, stream, split, t0, t1, tx, a, split, wait_limit);
}

template <bool kGated>
int launch_any(const char *where, const uint8_t *xq, const uint8_t *w0, const uint8_t *w1, const Args &a, cudaStream_t st) {
    if (a.M <= 16) return launch<16, kGated>(where, xq, w0, w1, a, st, kWaitLimit);
    if (a.M <= 32) return launch<32, kGated>(where, xq, w0, w1, a, st, kWaitLimit);
    if (a.M <= 64) return launch<64, kGated>(where, xq, w0, w1, a, st, kWaitLimit);
    if (a.M <= 128) return launch<128, kGated>(where, xq, w0, w1, a, st, kWaitLimit);
    return f8b::launch_tile(where, xq, w0, w1, a, st, kWaitLimit);
}

}  // namespace f8s

}  // namespace

}  // namespace qspec

using namespace qspec;

extern "C" int qspec_linear_fp8_block(const uint8_t *xq, const float *sa, int lds, const uint8_t *w8, const float *sw, int M,
                                      int N, int K, uint16_t *y_bf16, int ldy, int32_t *dev_status, qspec_stream_t stream) {
    if (!xq || !sa || !w8 || !sw || !y_bf16) return QSPEC_ERR_NULL;
    if (M < 1 || M > f8b::kMaxM || N < 1 || N > f8b::kMaxN || K < kGroup || K % kGroup || ldy < N || lds < M) return QSPEC_ERR_SHAPE;
    if (!aligned(xq, 16) || !aligned(w8, 16) || !aligned(sa, 4) || !aligned(sw, 4) || !aligned(y_bf16, 2))
        return QSPEC_ERR_ALIGN;
    int rc = check_device();
    if (rc) return rc;
    const f8b::Args a = {sa, sw, nullptr, y_bf16, nullptr, nullptr, dev_status, lds, M, N, K, ldy, 0};
    return f8s::launch_any<false>("qspec_linear_fp8_block", xq, w8, nullptr, a, as_cuda(stream));
}

extern "C" int qspec_gated_fp8_block(const uint8_t *xq, const float *sa, int lds, const uint8_t *w_gate, const float *s_gate,
                                     const uint8_t *w_up, const float *s_up, int M, int N, int K, uint8_t *hq, float *sh,
                                     int ldh, uint16_t *h_bf16, int ldy, int32_t *dev_status, qspec_stream_t stream) {
    if (!xq || !sa || !w_gate || !s_gate || !w_up || !s_up || (hq != nullptr) != (sh != nullptr) || (!hq && !h_bf16))
        return QSPEC_ERR_NULL;
    if (M < 1 || M > f8b::kMaxM || N < kGroup || N > f8b::kMaxN || N % kGroup || K < kGroup || K % kGroup || lds < M || (hq && ldh < M) || (h_bf16 && ldy < N))
        return QSPEC_ERR_SHAPE;
    if (!aligned(xq, 16) || !aligned(w_gate, 16) || !aligned(w_up, 16) || !aligned(sa, 4) || !aligned(s_gate, 4) ||
        !aligned(s_up, 4) || (hq && (!aligned(hq, 16) || !aligned(sh, 4))) || (h_bf16 && !aligned(h_bf16, 2)))
        return QSPEC_ERR_ALIGN;
    int rc = check_device();
    if (rc) return rc;
    const f8b::Args a = {sa, s_gate, s_up, h_bf16, hq, sh, dev_status, lds, M, N, K, ldy, ldh};
    return f8s::launch_any<true>("qspec_gated_fp8_block", xq, w_gate, w_up, a, as_cuda(stream));
}
