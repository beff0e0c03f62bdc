// 8-bit GEMM for few output tiles: Y = sum over K blocks of
// 2^(ex + ew) (Xq Wq^T), e4m3 operands with E8M0 block scales, bf16 out.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 multiplies each 32-channel piece of a row by
// the row's scale, so the block scales cost no vector instruction and no
// separate accumulator.  Lane l, r = l % 32, h = l / 32: A = row r, B = column
// r, 32 channels each; which channels a half holds does not matter as long as A
// and B agree and all of them have one scale.  D: column r, rows
// 8 (e / 4) + 4 h + e % 4.
// Rounding (pinned by the tests): the instruction adds products in groups of 8
// channels, dropping what lies below 2^-13 of the group's largest product, then
// adds the groups and the accumulator in fp32.  That is far below what e4m3 took
// from the inputs (2^-4 of a value); the alternative that keeps every bit, the
// bf16 instruction on widened values, runs at half the rate.
//
// One 32 x 32 RT tile per workgroup.  Its 8 waves take the K blocks in turn,
// each straight from global memory into registers (per block a lane reads 64
// contiguous bytes of its row, a row's two halves one 128-byte line), and their
// sums are joined through LDS in wave order, so the result does not depend on
// timing.  With few rows the weight's bytes are what bounds it.
#include "lynx_fp8.h"

namespace lynx {
namespace {

constexpr int kWaves = 8;

template <int RT>
__global__ __launch_bounds__(64 * kWaves) void gemm_fp8_split(
    const uint8_t* __restrict__ Xq, const uint32_t* __restrict__ Xs,
    const uint8_t* __restrict__ Wq, const uint8_t* __restrict__ Ws, uint16_t* __restrict__ Y,
    int M, int N, int K, int tiles_m) {
    __shared__ float part[kWaves][32][33];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int r = lane & 31, h = lane >> 5;
    const int m0 = int(blockIdx.x % tiles_m) * 32 * RT, n0 = int(blockIdx.x / tiles_m) * 32;
    const int blocks = (K + kFp8Block - 1) / kFp8Block;
    const int pitch = 4 * fp8_scale_words(K);

    // rows past the end read the last row; their results are not stored
    const uint8_t* b = Wq + size_t(min(n0 + r, N - 1)) * size_t(K) + 64 * h;
    const uint8_t* bs = Ws + size_t(n0 / kFp8Block) * size_t(pitch);
    const uint8_t* a[RT];
    const uint32_t* as[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        const int row = min(m0 + 32 * t + r, M - 1);
        a[t] = Xq + size_t(row) * size_t(K) + 64 * h;
        as[t] = Xs + row;
    }
    f32x16 acc[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) acc[t] = f32x16{};
    for (int kb = wave; kb < blocks; kb += kWaves) {
        const bool in = kb * kFp8Block + 64 * h < K;  // a last block of 64 has no second half
        i32x8 bf[2] = {}, af[RT][2] = {};
        if (in) {
#pragma unroll
            for (int s = 0; s < 2; ++s) {
                bf[s] = *reinterpret_cast<const i32x8*>(b + kb * kFp8Block + 32 * s);
#pragma unroll
                for (int t = 0; t < RT; ++t)
                    af[t][s] = *reinterpret_cast<const i32x8*>(a[t] + kb * kFp8Block + 32 * s);
            }
        }
        const int sb = bs[kb];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
            const int sa = int(as[t][size_t(kb >> 2) * size_t(M)] >> (8 * (kb & 3)));
#pragma unroll
            for (int s = 0; s < 2; ++s)
                acc[t] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(af[t][s], bf[s], acc[t],
                                                                         0, 0, 0, sa, 0, sb);
        }
    }
#pragma unroll
    for (int t = 0; t < RT; ++t) {
        if (t > 0) __syncthreads();
#pragma unroll
        for (int e = 0; e < 16; ++e) part[wave][8 * (e / 4) + 4 * h + e % 4][r] = acc[t][e];
        __syncthreads();
        const int row = threadIdx.x >> 4;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const int col = 2 * (threadIdx.x & 15) + j;
            float v = 0.f;
#pragma unroll
            for (int w = 0; w < kWaves; ++w) v += part[w][row][col];
            const int m = m0 + 32 * t + row, n = n0 + col;
            if (m < M && n < N)
                Y[size_t(m) * size_t(N) + n] =
                    __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
        }
    }
}

}  // namespace

lynx_status launch_gemm_fp8_split(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                            const uint8_t* Ws, uint16_t* Y, int M, int N, int K,
                            hipStream_t stream) {
    const uint32_t* xs = reinterpret_cast<const uint32_t*>(Xs);
    const int tn = (N + 31) / 32;
    if (M <= 32) {
        hipLaunchKernelGGL(gemm_fp8_split<1>, dim3(unsigned(tn)), dim3(64 * kWaves), 0, stream, Xq,
                           xs, Wq, Ws, Y, M, N, K, 1);
    } else {
        const int tm = (M + 63) / 64;
        hipLaunchKernelGGL(gemm_fp8_split<2>, dim3(unsigned(tm) * unsigned(tn)),
                           dim3(64 * kWaves), 0, stream, Xq, xs, Wq, Ws, Y, M, N, K, tm);
    }
    return launch_status();
}

}  // namespace lynx
