// attn_kv4.cu -- attention of the newest rows of every sequence over the 4-bit
// KV cache (draft steps and verify passes).
//
//   a_t = scale s_t (sum_d q_d c_td - z_t sum_d q_d),  p = softmax(a),
//   o = sum_t p_t s_t (c_t - z_t)
//
// First form: one CTA per (row, query head), one warp per cache position at a
// time with the head's D values spread over its lanes, running maximum and
// sum per warp, the warps joined at the end.
#include <cmath>

#include <cuda_fp16.h>

#include "qspec_device.cuh"
#include "qspec_host.h"

namespace qspec {

namespace {

namespace akv {

constexpr int kMaxR = QSPEC_MAX_GAMMA + 1;
constexpr int kThreads = 256, kWarps = kThreads / 32;

template <int D>
__global__ void __launch_bounds__(kThreads)
    simple_kernel(const uint16_t *__restrict__ q, int ldq, const uint8_t *__restrict__ kc,
                  const uint32_t *__restrict__ ks, const uint8_t *__restrict__ vc, const uint32_t *__restrict__ vs,
                  const int32_t *__restrict__ len, int R, int Hq, int H, int T, float scale, uint16_t *__restrict__ o,
                  int ldo, int32_t *st) {
    constexpr int E = D / 32;
    __shared__ float sm_m[kWarps], sm_l[kWarps], sm_o[kWarps][D];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int row = blockIdx.x, j = blockIdx.y, b = row / R, r = row - b * R, h = j / (Hq / H);
    pdl_launch_dependents();
    pdl_wait();
    const int n = len[b];
    if (n < 0 || n > T) {
        if (threadIdx.x == 0) flag(st, QSPEC_ERR_RANGE);
        return;
    }
    const int seen = n - R + r + 1;
    float qv[E], acc[E];
#pragma unroll
    for (int e = 0; e < E; ++e) {
        qv[e] = bf16_bits_to_float(q[(size_t)row * ldq + (size_t)j * D + lane * E + e]);
        acc[e] = 0.0f;
    }
    float m = -INFINITY, l = 0.0f;
    const size_t head = ((size_t)b * H + h) * T;
    for (int t = warp; t < seen; t += kWarps) {
        auto value = [&](const uint8_t *codes, uint32_t w, int e) {
            const int d = lane * E + e;
            const int c = (codes[(head + t) * (D / 2) + d / 2] >> (4 * (d & 1))) & 15;
            return __half2float(__ushort_as_half((uint16_t)(w & 0xFFFF))) *
                   ((float)c - __half2float(__ushort_as_half((uint16_t)(w >> 16))));
        };
        const uint32_t kw = ks[head + t], vw = vs[head + t];
        float a = 0.0f;
#pragma unroll
        for (int e = 0; e < E; ++e) a = fmaf(qv[e], value(kc, kw, e), a);
#pragma unroll
        for (int x = 16; x >= 1; x >>= 1) a += __shfl_xor_sync(0xffffffffu, a, x);
        a *= scale;
        const float m1 = fmaxf(m, a), f = expf(m - m1), p = expf(a - m1);
        m = m1;
        l = l * f + p;
#pragma unroll
        for (int e = 0; e < E; ++e) acc[e] = acc[e] * f + p * value(vc, vw, e);
    }
    if (lane == 0) {
        sm_m[warp] = m;
        sm_l[warp] = l;
    }
#pragma unroll
    for (int e = 0; e < E; ++e) sm_o[warp][lane * E + e] = acc[e];
    __syncthreads();
    float mm = -INFINITY, ll = 0.0f;
    for (int w = 0; w < kWarps; ++w) mm = fmaxf(mm, sm_m[w]);
    for (int w = 0; w < kWarps; ++w) ll += sm_l[w] > 0.0f ? sm_l[w] * expf(sm_m[w] - mm) : 0.0f;
    for (int d = threadIdx.x; d < D; d += kThreads) {
        float x = 0.0f;
        for (int w = 0; w < kWarps; ++w) x += sm_l[w] > 0.0f ? sm_o[w][d] * expf(sm_m[w] - mm) : 0.0f;
        o[(size_t)row * ldo + (size_t)j * D + d] = float_to_bf16_bits(ll > 0.0f ? x / ll : 0.0f);
    }
}

bool sizes_ok(int B, int R, int Hq, int H, int D) {
    return B >= 1 && R >= 1 && R <= kMaxR && H >= 1 && Hq >= H && Hq % H == 0 && (D == 64 || D == 128) &&
           (long long)B * R * Hq < (1LL << 28);
}

}  // namespace akv

}  // namespace

}  // namespace qspec

using namespace qspec;

extern "C" size_t qspec_attn_kv4_workspace_bytes(int B, int R, int Hq, int H, int D) {
    return akv::sizes_ok(B, R, Hq, H, D) ? 16 : 0;
}

extern "C" int qspec_attn_kv4(const uint16_t *q_bf16, int ldq, const uint8_t *k_codes, const uint32_t *k_sz,
                              const uint8_t *v_codes, const uint32_t *v_sz, const int32_t *len, int B, int R, int Hq,
                              int H, int T, int D, float scale, uint16_t *o_bf16, int ldo, void *workspace,
                              size_t ws_bytes, int32_t *dev_status, qspec_stream_t stream) {
    if (!q_bf16 || !k_codes || !k_sz || !v_codes || !v_sz || !len || !o_bf16 || !workspace) return QSPEC_ERR_NULL;
    if (!akv::sizes_ok(B, R, Hq, H, D) || T < 1 || !std::isfinite(scale) || ldq < (long long)Hq * D ||
        ldo < (long long)Hq * D)
        return QSPEC_ERR_SHAPE;
    if (ldq % 8 || ldo % 8 || !aligned(q_bf16, 16) || !aligned(o_bf16, 16) || !aligned(k_codes, 16) ||
        !aligned(v_codes, 16) || !aligned(k_sz, 4) || !aligned(v_sz, 4) || !aligned(len, 4) || !aligned(workspace, 16))
        return QSPEC_ERR_ALIGN;
    if (ws_bytes < qspec_attn_kv4_workspace_bytes(B, R, Hq, H, D)) return QSPEC_ERR_WORKSPACE;
    int rc = check_device();
    if (rc) return rc;
    auto kern = D == 128 ? akv::simple_kernel<128> : akv::simple_kernel<64>;
    return launch_pdl("qspec_attn_kv4", kern, dim3((unsigned)(B * R), (unsigned)Hq), dim3(akv::kThreads), 0,
                      as_cuda(stream), q_bf16, ldq, k_codes, k_sz, v_codes, v_sz, len, R, Hq, H, T, scale, o_bf16,
                      ldo, dev_status);
}
