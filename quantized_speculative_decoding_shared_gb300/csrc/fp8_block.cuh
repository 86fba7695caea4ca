// fp8_block.cuh -- what the products of E4M3 codes with a scale for each block
// of 128 share: their arguments, and the epilogue of the gated one.
#pragma once

#include <cuda_fp8.h>

#include "qspec_device.cuh"

namespace qspec {
namespace f8b {

constexpr int kMaxM = 1 << 22, kMaxN = 1 << 30;   // what the grids count

struct Args {
    const float *sa;             // [K / 128][lds] scales of the tokens
    const float *s0, *s1;        // [ceil(N / 128)][K / 128] scales of the weights (gated: gate, up)
    uint16_t *y;                 // bf16 output (gated: may be null)
    uint8_t *hq;                 // gated: E4M3 output and its scales [N / 128][ldh] (may be null)
    float *sh;
    int32_t *st;
    int lds, M, N, K, ldy, ldh;
};

// h = silu(g) u = g u / (1 + exp(-g)).  exp(-g) passes fp32 below -88.7: 1 / inf is the limit 0; a NaN stays one.
__device__ __forceinline__ float gated(float g, float u) { return __fdividef(g, 1.0f + __expf(-g)) * u; }

// A block's scale and what its codes are taken with: E4M3(v up inv), inv = 448 / (up max |v|), up = 2^96 where 448 / max
// |v| would pass fp32.  Within 2 x 2^-24 of v / s in the quotient.  A scale of 0 has the codes 0.
struct Quant {
    float s, inv, up;
    __device__ __forceinline__ explicit Quant(float amax) {
        up = amax < 1.0e-30f ? 7.9228162514264338e28f : 1.0f;
        s = __fdiv_rn(amax, 448.0f);
        inv = s > 0.0f ? __fdiv_rn(448.0f, amax * up) : 0.0f;
    }
};

// four codes, the first in the low byte
__device__ __forceinline__ uint32_t codes4(float a, float b, float c, float d) {
    const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
    const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
    return lo | hi << 16;
}

}  // namespace f8b
}  // namespace qspec
