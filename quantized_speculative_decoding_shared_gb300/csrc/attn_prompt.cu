// attn_prompt.cu -- causal attention of packed prompts, grouped heads.
//
//   a_ij = scale q_i . k_j for j <= i + Lk - Lq,  o_i = sum_j softmax(a_i)_j v_j
//
// First form: one CTA per (32 query rows of a sequence, query head), eight
// rows per warp, key tiles of 32 rows in shared memory, running maximum and sum.
#include <cmath>

#include "qspec_device.cuh"
#include "qspec_host.h"

namespace qspec {

namespace {

namespace apr {

constexpr int kThreads = 128, kTile = 32, kRowsPerWarp = 8;

template <int D>
__global__ void __launch_bounds__(kThreads)
    simple_kernel(const uint16_t *__restrict__ q, int ldq, const uint16_t *__restrict__ k, int ldk,
                  const uint16_t *__restrict__ v, int ldv, const int32_t *__restrict__ q_start,
                  const int32_t *__restrict__ k_start, int q_rows, int k_rows, int B, int Hq, int H, float scale,
                  uint16_t *__restrict__ o, int ldo, int32_t *st) {
    constexpr int E = D / 32;
    __shared__ float sq[kTile][D], sk[kTile][D + 1];
    __shared__ uint16_t sv[kTile][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = blockIdx.y, h = j / (Hq / H);
    pdl_launch_dependents();
    pdl_wait();
    // tile blockIdx.x of the sequences' 32-row tiles in order
    int left = blockIdx.x, b = 0, q0 = 0, q1 = 0, k0 = 0, k1 = 0;
    for (; b < B; ++b) {
        q0 = q_start[b], q1 = q_start[b + 1], k0 = k_start[b], k1 = k_start[b + 1];
        if (q0 < 0 || q1 < q0 || q1 > q_rows || k0 < 0 || k1 < k0 || k1 > k_rows) {
            if (threadIdx.x == 0) flag(st, QSPEC_ERR_RANGE);
            continue;
        }
        const int tiles = (q1 - q0 + kTile - 1) / kTile;
        if (left < tiles) break;
        left -= tiles;
    }
    if (blockIdx.x == 0 && j == 0)                 // the sequences after this tile's are checked too
        for (int c = threadIdx.x; c < B; c += kThreads)
            if (q_start[c] < 0 || q_start[c + 1] < q_start[c] || q_start[c + 1] > q_rows || k_start[c] < 0 ||
                k_start[c + 1] < k_start[c] || k_start[c + 1] > k_rows)
                flag(st, QSPEC_ERR_RANGE);
    if (b == B) return;
    const int lq = q1 - q0, lk = k1 - k0, r0 = left * kTile;
    for (int e = threadIdx.x; e < kTile * D; e += kThreads) {
        const int i = e / D, d = e - i * D;
        sq[i][d] = r0 + i < lq ? bf16_bits_to_float(q[(size_t)(q0 + r0 + i) * ldq + (size_t)j * D + d]) : 0.0f;
    }
    float m[kRowsPerWarp], l[kRowsPerWarp], acc[kRowsPerWarp][E];
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
        m[i] = -INFINITY;
        l[i] = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[i][e] = 0.0f;
    }
    const int end = min(lk, min(r0 + kTile, lq) + lk - lq);          // keys that any row of the tile sees
    for (int t0 = 0; t0 < end; t0 += kTile) {
        __syncthreads();
        for (int e = threadIdx.x; e < kTile * D; e += kThreads) {
            const int i = e / D, d = e - i * D;
            const bool in = t0 + i < end;
            sk[i][d] = in ? bf16_bits_to_float(k[(size_t)(k0 + t0 + i) * ldk + (size_t)h * D + d]) : 0.0f;
            sv[i][d] = in ? v[(size_t)(k0 + t0 + i) * ldv + (size_t)h * D + d] : (uint16_t)0;
        }
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kRowsPerWarp; ++i) {
            const int r = warp * kRowsPerWarp + i, seen = r0 + r + lk - lq + 1;   // keys 0 .. seen - 1
            float a = 0.0f;
#pragma unroll 16
            for (int d = 0; d < D; ++d) a = fmaf(sq[r][d], sk[lane][d], a);
            a = t0 + lane < min(seen, end) ? a * scale : -INFINITY;
            float mt = a;
#pragma unroll
            for (int x = 16; x >= 1; x >>= 1) mt = fmaxf(mt, __shfl_xor_sync(0xffffffffu, mt, x));
            const float m1 = fmaxf(m[i], mt);
            const float ref = m1 > -INFINITY ? m1 : 0.0f;
            const float f = expf(m[i] - ref), p = expf(a - ref);
            float ps = p;
#pragma unroll
            for (int x = 16; x >= 1; x >>= 1) ps += __shfl_xor_sync(0xffffffffu, ps, x);
            m[i] = m1;
            l[i] = l[i] * f + ps;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[i][e] *= f;
            for (int t = 0; t < min(kTile, min(seen, end) - t0); ++t) {
                const float pt = __shfl_sync(0xffffffffu, p, t);
#pragma unroll
                for (int e = 0; e < E; ++e) acc[i][e] = fmaf(pt, bf16_bits_to_float(sv[t][lane + 32 * e]), acc[i][e]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kRowsPerWarp; ++i) {
        const int r = r0 + warp * kRowsPerWarp + i;
        if (r >= lq) continue;
#pragma unroll
        for (int e = 0; e < E; ++e)
            o[(size_t)(q0 + r) * ldo + (size_t)j * D + lane + 32 * e] =
                float_to_bf16_bits(l[i] > 0.0f ? acc[i][e] / l[i] : 0.0f);
    }
}

}  // namespace apr

}  // namespace

}  // namespace qspec

using namespace qspec;

extern "C" int qspec_attn_prompt(const uint16_t *q_bf16, int ldq, const uint16_t *k_bf16, int ldk,
                                 const uint16_t *v_bf16, int ldv, const int32_t *q_start, const int32_t *k_start,
                                 int q_rows, int k_rows, int B, int Hq, int H, int D, float scale, uint16_t *o_bf16,
                                 int ldo, int32_t *dev_status, qspec_stream_t stream) {
    if (!q_start || !k_start || (q_rows > 0 && (!q_bf16 || !o_bf16)) || (k_rows > 0 && (!k_bf16 || !v_bf16)))
        return QSPEC_ERR_NULL;
    if (q_rows < 0 || k_rows < 0 || B < 1 || H < 1 || Hq < H || Hq % H || Hq > 65535 || (D != 64 && D != 128) ||
        !std::isfinite(scale) || ldq < (long long)Hq * D || ldo < (long long)Hq * D || ldk < (long long)H * D ||
        ldv < (long long)H * D)
        return QSPEC_ERR_SHAPE;
    if ((ldq | ldk | ldv | ldo) % 8 || !aligned(q_bf16, 16) || !aligned(k_bf16, 16) || !aligned(v_bf16, 16) ||
        !aligned(o_bf16, 16) || !aligned(q_start, 4) || !aligned(k_start, 4))
        return QSPEC_ERR_ALIGN;
    int rc = check_device();
    if (rc || q_rows == 0) return rc;
    const long long tiles = (long long)q_rows / apr::kTile + B;
    if (tiles >= (1LL << 31)) return QSPEC_ERR_SHAPE;
    auto kern = D == 128 ? apr::simple_kernel<128> : apr::simple_kernel<64>;
    return launch_pdl("qspec_attn_prompt", kern, dim3((unsigned)tiles, (unsigned)Hq), dim3(apr::kThreads), 0,
                      as_cuda(stream), q_bf16, ldq, k_bf16, ldk, v_bf16, ldv, q_start, k_start, q_rows, k_rows, B, Hq,
                      H, scale, o_bf16, ldo, dev_status);
}
