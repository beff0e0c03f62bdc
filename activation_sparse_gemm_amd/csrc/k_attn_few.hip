// Attention of few query rows to a key head, as a kernel of its own; and side by side with tiles
// of 128 rows, for a prefix that the batch shares: all sequences' rows together on the prefix, each
// sequence's rows on its own keys.  48 tokens on a prefix of 8192 and up to 512 keys of their own,
// 32/8 x 128: 27 us, and 5 for the join (side by side saved 4 of 43 us, cutting the prefix for it 8).
#include "lynx_attn_few.h"
#include "lynx_attn_tile.h"

namespace lynx {
namespace {

template <int DP, bool LSE, bool CAUSAL>
__global__ __launch_bounds__(256, 2) void attn_few_kernel(const AttnArgs A) {
    __shared__ __attribute__((aligned(1024))) char smem[65536];
    __shared__ float stat[3][4][32];
    attn_few<DP, LSE, CAUSAL>(A, int(blockIdx.x), smem, stat);
}

// The first tile_grid workgroups (a multiple of 8) take the tiles, which take longest.
template <int DP, bool LSE, bool CAUSAL>
__global__ __launch_bounds__(256, 2) void attn_pair_kernel(const AttnArgs tile, int tile_grid, const AttnArgs few) {
    __shared__ __attribute__((aligned(1024))) char smem[65536];
    __shared__ float stat[3][4][32];
    const int block = int(blockIdx.x);
    if (block < tile_grid) attn_tile<DP, LSE, false>(tile, block, smem);
    else attn_few<DP, LSE, CAUSAL>(few, block - tile_grid, smem, stat);
}

}  // namespace

lynx_status launch_attn_few(const AttnArgs& a, int grid, hipStream_t stream) {
    const dim3 g{unsigned(grid)}, block{256};
    auto go = [&](auto dp, auto lse, auto causal) {
        hipLaunchKernelGGL((attn_few_kernel<dp, lse, causal>), g, block, 0, stream, a);
    };
    attn_variant(a, go);
    return launch_status();
}

lynx_status launch_attn_pair(const AttnArgs& tile, int tile_grid, const AttnArgs& few, int few_grid,
                             hipStream_t stream) {
    const dim3 g{unsigned(tile_grid + few_grid)}, block{256};
    auto go = [&](auto dp, auto lse, auto causal) {
        hipLaunchKernelGGL((attn_pair_kernel<dp, lse, causal>), g, block, 0, stream, tile, tile_grid, few);
    };
    attn_variant(few, go);
    return launch_status();
}

}  // namespace lynx
