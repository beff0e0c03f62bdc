// 8-bit GEMM for at most 16 rows (single tokens, conditioning vectors): the weight's
// bytes are what bounds it.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 multiplies each 32-channel piece of a row by
// the row's scale, so the block scales cost no vector instruction and no separate
// accumulator.  Lane l, r = l % 16, q = l / 16: A = row r of X, B = row r of W's
// tile, 32 channels each; which channels a q holds does not matter as long as A and
// B agree and all of them have one scale.  D: column r, rows 4 q .. 4 q + 3.
// Rounding (pinned by the tests): the instruction adds products in groups of 8
// channels, dropping what lies below 2^-13 of the group's largest product, then
// adds the groups and the accumulator in fp32.  That is far below what e4m3 took
// from the inputs (2^-4 of a value); the alternative that keeps every bit, the
// bf16 instruction on widened values, runs at half the rate.
//
// A workgroup takes 16 columns; its 8 waves take the K blocks in turn, straight
// from global memory into registers: per 16 rows and block two loads of 16 bytes a
// lane, each 64 contiguous bytes of 16 rows, three blocks under way.  From HBM, in us
// (one block ahead, 16 waves): 2 x 3072 -> 18432 12.8 = 4.4 TB/s (14.4, 13.8); 1 x 12288
// -> 3072 11.5 (14.1, 11.5); from the cache the first takes 11.2 (12.3, 12.3).  The
// waves' sums are joined through LDS in wave order, so the result does not depend on
// timing.
//
// QUANT reads bf16 X and quantises it first, as lynx_quantize_fp8 does, into LDS: 16
// lanes a row's block.  Every workgroup repeats that, so it is used where X is small
// (fp8_fuse); there it takes the place of a second kernel and of the
// 8-bit copy in memory.
#include "lynx_fp8.h"

namespace lynx {
namespace {

typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kWaves = 8;
constexpr int kDepth = 3;  // blocks of a wave that are under way

template <bool QUANT>
__global__ __launch_bounds__(64 * kWaves) void gemm_fp8_few(
    const void* __restrict__ X, const uint32_t* __restrict__ Xs, const uint8_t* __restrict__ Wq,
    const uint32_t* __restrict__ Ws, uint16_t* __restrict__ Y, int M, int N, int K) {
    __shared__ float part[kWaves][16][17];
    // the rows' quantised blocks [block][row], 16-byte chunks swizzled by the row, and
    // their scales: at most M K + 64 M bytes, and a scale for each 128 of them
    constexpr int kX = QUANT ? kFewQuant + 64 * kFewRows : 16;
    __shared__ __attribute__((aligned(16))) char xq[kX];
    __shared__ uint8_t xs[QUANT ? kX / kFp8Block : 16];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int r = lane & 15, q = lane >> 4;
    const int n0 = int(blockIdx.x) * 16;
    const int blocks = (K + kFp8Block - 1) / kFp8Block;
    const int words = fp8_scale_words(K);

    // rows past the end read the last row; their results are not stored
    const int xrow = min(r, M - 1);
    const uint8_t* a = static_cast<const uint8_t*>(X) + size_t(xrow) * size_t(K) + 16 * q;
    const int wrow = min(n0 + r, N - 1);
    const uint8_t* b = Wq + size_t(wrow) * size_t(K) + 16 * q;
    const uint32_t* bs = Ws + size_t(wrow / kFp8Block) * size_t(words);
    struct Block {
        i32x4 a[2], b[2];
        uint32_t sa, sb;
    };
    auto load = [&](int kb, Block& o) {
        const int off = kb * kFp8Block;
        const bool upper = off + 64 < K;  // a last block of 64 channels has no upper half: zeros
        o.b[0] = *reinterpret_cast<const i32x4*>(b + off);
        o.b[1] = upper ? *reinterpret_cast<const i32x4*>(b + off + 64) : i32x4{};
        o.sb = bs[kb >> 2];
        if constexpr (!QUANT) {
            o.a[0] = *reinterpret_cast<const i32x4*>(a + off);
            o.a[1] = upper ? *reinterpret_cast<const i32x4*>(a + off + 64) : i32x4{};
            o.sa = Xs[size_t(kb >> 2) * size_t(M) + xrow];
        }
    };
    f32x4 acc = {};
    auto multiply = [&](int kb, const Block& o) {
        const int shift = 8 * (kb & 3);
        i32x4 lo = o.a[0], hi = o.a[1];
        int sa = int(o.sa >> shift);
        if constexpr (QUANT) {
            const char* p = xq + (kb * M + xrow) * kFp8Block;
            lo = *reinterpret_cast<const i32x4*>(p + 16 * (q ^ fp8_swz(xrow)));
            hi = *reinterpret_cast<const i32x4*>(p + 16 * ((4 + q) ^ fp8_swz(xrow)));
            sa = xs[kb * M + xrow];
        }
        const i32x8 va = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        const i32x8 vb = __builtin_shufflevector(o.b[0], o.b[1], 0, 1, 2, 3, 4, 5, 6, 7);
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(va, vb, acc, 0, 0, 0, sa, 0,
                                                               int(o.sb >> shift));
    };
    Block ring[kDepth];
#pragma unroll
    for (int i = 0; i < kDepth; ++i)
        if (wave + i * kWaves < blocks) load(wave + i * kWaves, ring[i]);
    if constexpr (QUANT) {
        const int l16 = lane & 15;
        for (int u = wave * 4 + q; u < M * blocks; u += 4 * kWaves) {
            const int row = u % M, blk = u / M;
            const int c = blk * kFp8Block + 8 * l16;
            u32x4 v = {0, 0, 0, 0};
            if (c < K)
                v = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(X) +
                                                    size_t(row) * size_t(K) + c);
            const uint32_t byte = fp8_scale_byte(row16_max(fp8_amax8(v)));
            const float div = fp8_divisor(byte);
            *reinterpret_cast<u32x2*>(xq + u * kFp8Block + 16 * ((l16 >> 1) ^ fp8_swz(row)) +
                                      8 * (l16 & 1)) =
                u32x2{fp8_pack4(v[0], v[1], div), fp8_pack4(v[2], v[3], div)};
            if (l16 == 0) xs[u] = uint8_t(byte);
        }
        __syncthreads();
    }
    for (int kb = wave; kb < blocks; kb += kDepth * kWaves) {
#pragma unroll
        for (int i = 0; i < kDepth; ++i) {
            const int at = kb + i * kWaves;
            if (at >= blocks) break;
            multiply(at, ring[i]);
            if (at + kDepth * kWaves < blocks) load(at + kDepth * kWaves, ring[i]);
        }
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) part[wave][4 * q + e][r] = acc[e];
    __syncthreads();
    if (threadIdx.x < 256) {
        const int row = threadIdx.x >> 4, col = threadIdx.x & 15;
        float v = 0.f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v += part[w][row][col];
        if (row < M && n0 + col < N)
            Y[size_t(row) * size_t(N) + n0 + col] =
                __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
    }
}

}  // namespace

lynx_status launch_gemm_fp8_few(const void* X, const uint8_t* Xs, const uint8_t* Wq,
                                const uint8_t* Ws, uint16_t* Y, int M, int N, int K,
                                hipStream_t stream) {
    const dim3 grid(unsigned((N + 15) / 16));
    const uint32_t *xs = reinterpret_cast<const uint32_t*>(Xs),
                   *ws = reinterpret_cast<const uint32_t*>(Ws);
    if (Xs)
        hipLaunchKernelGGL(gemm_fp8_few<false>, grid, dim3(64 * kWaves), 0, stream, X, xs, Wq, ws, Y,
                           M, N, K);
    else
        hipLaunchKernelGGL(gemm_fp8_few<true>, grid, dim3(64 * kWaves), 0, stream, X, xs, Wq, ws, Y,
                           M, N, K);
    return launch_status();
}

}  // namespace lynx
