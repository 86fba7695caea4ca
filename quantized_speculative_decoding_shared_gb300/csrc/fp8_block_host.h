// fp8_block_host.h -- the kernels behind the products of E4M3 codes with block scales.
#pragma once

#include <algorithm>
#include <mutex>

#include "fp8_block.cuh"
#include "qspec_host.h"

namespace qspec {
namespace f8b {

// wait_limit, stall: as in qspec_host.h's launches of the other tensor-core kernels.
// Many tokens (fp8_block_tile.cu); w1: the up projection's weights of the gated product, else null.
int launch_tile(const char *where, const uint8_t *xq, const uint8_t *w0, const uint8_t *w1, const Args &a, cudaStream_t stream,
                uint32_t wait_limit, int stall);

// CTAs of a kernel (`per` to an SM) that the device runs at once in clusters of each size, a whole number of clusters
// (0: none).
struct Resident {
    int ctas[kMaxSplit + 1];
};
inline Resident ask_resident(const void *kern, int threads, size_t smem, bool max_carveout, int per) {
    Resident r = {};
    const int slots = sm_count() * per;
    r.ctas[1] = slots;
    if (smem_limit_once(kern, (int)smem, max_carveout)) return r;
    for (int c = 2; c <= kMaxSplit; ++c) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3((unsigned)(slots / c * c));
        cfg.blockDim = dim3((unsigned)threads);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute attr[1];
        attr[0].id = cudaLaunchAttributeClusterDimension;
        attr[0].val.clusterDim.x = (unsigned)c;
        attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
        cfg.attrs = attr;
        cfg.numAttrs = 1;
        int clusters = 0;
        if (cudaOccupancyMaxActiveClusters(&clusters, kern, &cfg) != cudaSuccess) {
            cudaGetLastError();
            clusters = 0;
        }
        r.ctas[c] = std::min(clusters * c, slots / c * c);
    }
    return r;
}
// Asked once for each device (the questions take some microseconds); Kernel: a type with the kernel's address, threads,
// shared memory (and whether it wants all there is as such) and CTAs per SM.
template <class Kernel>
Resident resident() {
    constexpr int kDevices = 64;
    static Resident known[kDevices];
    static std::once_flag once[kDevices];
    int dev = 0;
    cudaGetDevice(&dev);
    const auto ask = [] { return ask_resident(Kernel::address(), Kernel::threads, Kernel::smem, Kernel::carveout, Kernel::per); };
    if (dev < 0 || dev >= kDevices) return ask();
    std::call_once(once[dev], [&] { known[dev] = ask(); });
    return known[dev];
}

}  // namespace f8b
}  // namespace qspec
