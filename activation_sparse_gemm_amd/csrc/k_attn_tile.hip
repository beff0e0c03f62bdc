// Attention over tiles of 128 query rows, as a kernel of its own.
#include "lynx_attn_tile.h"

namespace lynx {
namespace {

template <int DP, bool LSE, bool CAUSAL>
__global__ __launch_bounds__(256, 2) void attn_tile_kernel(const AttnArgs A) {
    __shared__ __attribute__((aligned(1024))) char smem[65536];
    attn_tile<DP, LSE, CAUSAL>(A, int(blockIdx.x), smem);
}

}  // namespace

lynx_status launch_attn_tile(const AttnArgs& a, int grid, hipStream_t stream) {
    const dim3 g{unsigned(grid)}, block{256};
    auto go = [&](auto dp, auto lse, auto causal) {
        hipLaunchKernelGGL((attn_tile_kernel<dp, lse, causal>), g, block, 0, stream, a);
    };
    attn_variant(a, go);
    return launch_status();
}

}  // namespace lynx
