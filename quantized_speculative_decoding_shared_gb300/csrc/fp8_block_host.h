// fp8_block_host.h -- the kernels behind the products of E4M3 codes with block scales.
#pragma once

#include "fp8_block.cuh"
#include "qspec_host.h"

namespace qspec {
namespace f8b {

// wait_limit, stall: as in qspec_host.h's launches of the other tensor-core kernels.
// Many tokens (fp8_block_tile.cu); w1: the up projection's weights of the gated product, else null.
int launch_tile(const char *where, const uint8_t *xq, const uint8_t *w0, const uint8_t *w1, const Args &a, cudaStream_t stream,
                uint32_t wait_limit, int stall);

}  // namespace f8b
}  // namespace qspec
