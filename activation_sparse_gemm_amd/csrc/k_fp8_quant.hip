// Quantisers of the 8-bit layer: bf16 activations and weights to e4m3 with one
// power-of-two scale per block of 128 (layouts in lynx.h).
//
// Both read each input once, keep it in registers while the block's largest
// magnitude is found, and write each output once, so that HBM traffic (3 bytes
// per element) is what bounds them.
#include "lynx_fp8.h"

namespace lynx {
namespace {

__device__ __forceinline__ u32x2 quant8(const u32x4& v, float divisor) {
    return u32x2{fp8_pack4(v[0], v[1], divisor), fp8_pack4(v[2], v[3], divisor)};
}

// Activations.  A wave takes 512 channels (one scale word) of 2 consecutive
// rows: lane l holds channels 8l .. 8l+7, so a scale's 128 channels are the 16
// lanes of a DPP row.  9216 x 12288: 58.8 us (5.8 TB/s); 1 row a wave 61.3, 4 rows
// 59.9, 8 rows 63.3; 4096 x 3072: 8.8 us, 9.2, 8.5 and 9.2.
constexpr int kRows = 2;

__global__ __launch_bounds__(256) void quantize_fp8_kernel(const uint16_t* __restrict__ X,
                                                            uint8_t* __restrict__ q,
                                                            uint32_t* __restrict__ scale, int M,
                                                            int K, int words) {
    const int lane = threadIdx.x & 63;
    const int unit = __builtin_amdgcn_readfirstlane(int(blockIdx.x * 4 + (threadIdx.x >> 6)));
    const int word = unit % words;
    const int row0 = unit / words * kRows;
    if (row0 >= M) return;
    const int c = word * 512 + lane * 8;
    const bool in = c < K;  // K % 64 == 0: a lane's 8 channels are inside or outside together
    u32x4 v[kRows];
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        v[u] = u32x4{0, 0, 0, 0};
        if (in && row0 + u < M)
            v[u] = *reinterpret_cast<const u32x4*>(X + size_t(row0 + u) * size_t(K) + c);
    }
    uint32_t mine = 0;
#pragma unroll
    for (int u = 0; u < kRows; ++u) {
        const uint32_t byte = fp8_scale_byte(row16_max(fp8_amax8(v[u])));
        const u32x2 w = quant8(v[u], fp8_divisor(byte));
        if (in && row0 + u < M)
            *reinterpret_cast<u32x2*>(q + size_t(row0 + u) * size_t(K) + c) = w;
        const uint32_t sw = fp8_scale_word(byte);
        if (lane == u) mine = sw;
    }
    if (lane < kRows && row0 + lane < M) scale[size_t(word) * size_t(M) + row0 + lane] = mine;
}

// Weights: a workgroup takes a block of 128 rows x 128 channels; thread t holds
// channels 8 (t % 16) .. of rows t / 16 + 16 j.
__global__ __launch_bounds__(256) void quantize_fp8_weight_kernel(const uint16_t* __restrict__ W,
                                                                   uint8_t* __restrict__ q,
                                                                   uint8_t* __restrict__ scale,
                                                                   int N, int K, int blocks,
                                                                   int pitch) {
    __shared__ uint32_t part[4];
    const int t = threadIdx.x;
    const int kb = blockIdx.x % blocks, nb = blockIdx.x / blocks;
    const int c = kb * kFp8Block + (t & 15) * 8, r0 = nb * kFp8Block + (t >> 4);
    const bool in = c < K;
    u32x4 v[8];
    uint32_t m = 0;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        v[j] = u32x4{0, 0, 0, 0};
        if (in && r0 + 16 * j < N)
            v[j] = *reinterpret_cast<const u32x4*>(W + size_t(r0 + 16 * j) * size_t(K) + c);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) m = max(m, fp8_amax8(v[j]));
    m = row16_max(m);
    m = max(max(uint32_t(__builtin_amdgcn_readlane(int(m), 0)),
                uint32_t(__builtin_amdgcn_readlane(int(m), 16))),
            max(uint32_t(__builtin_amdgcn_readlane(int(m), 32)),
                uint32_t(__builtin_amdgcn_readlane(int(m), 48))));
    if ((t & 63) == 0) part[t >> 6] = m;
    __syncthreads();
    const uint32_t byte = fp8_scale_byte(max(max(part[0], part[1]), max(part[2], part[3])));
    const float div = fp8_divisor(byte);
#pragma unroll
    for (int j = 0; j < 8; ++j)
        if (in && r0 + 16 * j < N)
            *reinterpret_cast<u32x2*>(q + size_t(r0 + 16 * j) * size_t(K) + c) = quant8(v[j], div);
    // the last block of a row also fills the unused places of its last word
    const int n = kb == blocks - 1 ? pitch - kb : 1;
    if (t < n) scale[size_t(nb) * size_t(pitch) + kb + t] = uint8_t(t == 0 ? byte : kScaleOne);
}

}  // namespace

lynx_status launch_quantize_fp8(const uint16_t* X, int M, int K, uint8_t* q, uint8_t* scale,
                                hipStream_t stream) {
    const int words = fp8_scale_words(K);
    uint32_t* s = reinterpret_cast<uint32_t*>(scale);
    const dim3 grid(unsigned((int64_t((M + kRows - 1) / kRows) * words + 3) / 4));
    hipLaunchKernelGGL(quantize_fp8_kernel, grid, dim3(256), 0, stream, X, q, s, M, K, words);
    return launch_status();
}

lynx_status launch_quantize_fp8_weight(const uint16_t* W, int N, int K, uint8_t* q,
                                       uint8_t* scale, hipStream_t stream) {
    const int blocks = (K + kFp8Block - 1) / kFp8Block;
    const int nb = (N + kFp8Block - 1) / kFp8Block;
    hipLaunchKernelGGL(quantize_fp8_weight_kernel, dim3(unsigned(blocks) * unsigned(nb)), dim3(256),
                       0, stream, W, q, scale, N, K, blocks, 4 * fp8_scale_words(K));
    return launch_status();
}

}  // namespace lynx
