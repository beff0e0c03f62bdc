// 8-bit GEMM for a middling number of output tiles: too few 128 x 128 tiles to
// fill the chip, more rows than the K-split kernel's registers serve well.
//
// A workgroup of KG groups of 4 waves takes one tile of 32 RM x 32 CN outputs; group
// g takes the K blocks g, g + KG, ...  A step is KG blocks: 128-byte rows of X and W
// (swizzled) and the rows' scale words, moved by DMA into a ring of SLOTS slots, so
// that SLOTS - 1 steps are in flight: such a tile's arithmetic is short, and what
// bounds it is how many bytes a compute unit keeps under way.  Per step a wait, a
// barrier, the next loads, 2 (RM + CN) LDS reads and RM CN
// v_mfma_scale_f32_16x16x128_f8f6f4 a wave (matrix operand A = W, B = X; lane l, r =
// l % 16, q = l / 16: row r of each, 16-byte chunks q and 4 + q of a block; D: row r of
// X, rows 4 q .. 4 q + 3 of W).  Channels past K are loaded again from inside the row:
// the upper half of a last block of 64 is zeroed in W, blocks that fill up a step are
// weighted 2^-127 in both operands, whose products are zero in fp32.  (A lane's
// scale is that of the instruction's channels 32 q .. 32 q + 31, not of the lane's own
// two chunks: the scales of lanes q >= 2 could mask the upper half as well, as
// k_gemm_fp8.hip does.)  The groups' sums are joined through LDS in order.
//
// QUANT reads bf16 X and quantises it on the way, as lynx_quantize_fp8 does: a step's
// rows land as they are (256 bytes a block) and 16 lanes turn a row's block into its
// values and scale, in LDS, before the fragments are read (a second barrier).  Every
// column of tiles repeats that; it saves a kernel and the 8-bit copy's way through
// memory.
#include "lynx_fp8.h"
#include "lynx_tile.h"

namespace lynx {
namespace {

template <int RM, int CN, int KG, int SLOTS, bool QUANT>
__global__ __launch_bounds__(256 * KG) void gemm_fp8_mid(
    const void* __restrict__ X, const uint8_t* __restrict__ Xs,
    const uint8_t* __restrict__ Wq, const uint32_t* __restrict__ Ws, uint16_t* __restrict__ Y,
    int M, int N, int K) {
    constexpr int TM = 32 * RM, TN = 32 * CN;       // waves 2 x 2 of 16 RM x 16 CN
    constexpr int kX = TM * (QUANT ? 256 : 128), kW = TN * 128;
    constexpr int kGroup = kX + kW + (QUANT ? 0 : 1024);  // one block: + a scale word per row of X
    constexpr int kSlot = KG * kGroup;
    // W's scale word (a tile's columns lie in one scale block) comes with the step, behind
    // X's, by wave 3, where the step is short: a scalar load under way makes every wait for
    // LDS reads a wait for it too.  64 x 12288 -> 3072 14.0 us, 15.1 with scalar loads; but
    // 1000 x 12288 -> 3072 53.2 and 51.7, QUANT 333 x 1024 -> 1024 6.4 and 6.2.
    constexpr bool kStepW = !QUANT && RM * CN <= 4;
    // per wave and step
    constexpr int kDmaX = QUANT ? 2 * RM : RM, kDmaW = CN, kDma = kDmaX + kDmaW + (QUANT ? 0 : 1);
    constexpr int kJoin = (KG - 1) * TM * TN * 4;
    constexpr int kQ = QUANT ? TM * 128 + TM : 0;         // a group's quantised block and scales
    constexpr int kLds = SLOTS * kSlot + KG * kQ;
    static_assert(TM <= 128 && TN <= 128 && kLds <= 160 * 1024 && kJoin <= SLOTS * kSlot, "LDS budget");
    static_assert((SLOTS - 2) * kDma < 64, "vmcnt range");
    __shared__ __attribute__((aligned(1024))) char smem[kLds];

    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int wave = wid & 3, group = wid >> 2;
    const int r = lane & 15, q = lane >> 4;
    const int wm = wave & 1, wn = wave >> 1;
    const int tiles_m = (M + TM - 1) / TM, tiles_n = (N + TN - 1) / TN;
    int tm, tn;
    tile_of(blockIdx.x, tiles_m, tiles_n, tm, tn);
    const int blocks = (K + kFp8Block - 1) / kFp8Block;
    const int steps = (blocks + KG - 1) / KG;
    const int words = fp8_scale_words(K);
    const int nblocks = (N + kFp8Block - 1) / kFp8Block;

    const uint32_t lds0 = lds_addr(smem) + uint32_t(group * kGroup);
    const i32x4 rsX = make_rsrc(X, uint32_t(M) * uint32_t(K) * (QUANT ? 2u : 1u));
    const i32x4 rsW = make_rsrc(Wq, uint32_t(N) * uint32_t(K));
    const bool wscale = kStepW && wave == 3;
    const i32x4 rsS = wscale ? make_rsrc(Ws, uint32_t(nblocks) * uint32_t(words) * 4u)
                             : make_rsrc(Xs, uint32_t(words) * uint32_t(M) * 4u);
    const uint32_t wordS = wscale ? 4u : uint32_t(M) * 4u;  // from a word to the next
    // DMA instruction j of wave w moves rows 8 w + l/8 + 32 j, lane l's 16 bytes the
    // chunk that the row's swizzle puts there (the same for every j)
    const int lrow = 8 * wave + (lane >> 3);
    const int chunk = (lane & 7) ^ fp8_swz(lrow);
    // (QUANT: X's rows are 256 bytes, unswizzled: rows 4 w + l/16 + 16 j)
    const int qrow = 4 * wave + (lane >> 4);
    const uint32_t vx = QUANT ? uint32_t(tm * TM + qrow) * uint32_t(2 * K) + uint32_t(16 * r)
                              : uint32_t(tm * TM + lrow) * uint32_t(K) + uint32_t(16 * chunk);
    const uint32_t vw = uint32_t(tn * TN + lrow) * uint32_t(K) + uint32_t(16 * chunk);
    // rows past the end take the last row's words (the word's offset is not range checked)
    const uint32_t vs = wscale ? uint32_t(tn * TN / kFp8Block * words) * 4u
                               : uint32_t(min(tm * TM + (64 * wave) % TM + lane, M - 1)) * 4u;
    auto load = [&](int step, int slot) {  // past the last step: the last block again
        const uint32_t base = lds0 + uint32_t(slot * kSlot);
        const int kb = min(step * KG + group, blocks - 1);
        const uint32_t back = kb * kFp8Block + 64 < K || chunk < 4 ? 0u : 64u;
        const uint32_t off = uint32_t(kb) * kFp8Block;
#pragma unroll
        for (int j = 0; j < kDmaX; ++j) {
            if constexpr (QUANT)
                dma16(base + 1024 * (wave + 4 * j),
                      vx - (kb * kFp8Block + 64 < K || r < 8 ? 0u : 128u) +
                          uint32_t(16 * j) * uint32_t(2 * K), rsX, 2 * off);
            else
                dma16(base + 1024 * (wave + 4 * j), vx - back + uint32_t(32 * j) * uint32_t(K), rsX,
                      off);
        }
#pragma unroll
        for (int j = 0; j < kDmaW; ++j)
            dma16(base + kX + 1024 * (wave + 4 * j), vw - back + uint32_t(32 * j) * uint32_t(K), rsW,
                  off);
        if constexpr (!QUANT)
            dma4(base + kX + kW + 256 * wave, vs, rsS, uint32_t(kb >> 2) * wordS);
    };
#pragma unroll
    for (int s = 0; s < SLOTS - 1; ++s) load(s, s);

    static_assert(128 % TN == 0, "a tile's columns lie in one scale block of W");
    const uint32_t* wsp = Ws + size_t(tn * TN / kFp8Block) * size_t(words);
    uint32_t ws = 0;
    if constexpr (!kStepW) ws = wsp[min(group >> 2, words - 1)];
    const int row0 = tm * TM + wm * 16 * RM, col0 = tn * TN + wn * 16 * CN;
    const int sw = fp8_swz(r);
    char* const xq = smem + SLOTS * kSlot + group * kQ;      // QUANT: the group's values ...
    uint8_t* const xs = reinterpret_cast<uint8_t*>(xq + TM * 128);  // ... and scales
    const int offX = (QUANT ? 0 : group * kGroup) + (wm * 16 * RM + r) * 128;
    const int offW = group * kGroup + kX + (wn * 16 * CN + r) * 128;
    const int offS = group * kGroup + kX + kW + (wm * 16 * RM + r) * 4;
    f32x4 acc[RM][CN];
#pragma unroll
    for (int i = 0; i < RM; ++i)
#pragma unroll
        for (int j = 0; j < CN; ++j) acc[i][j] = f32x4{};

    int slot = 0;
    for (int step = 0; step < steps; ++step) {
        const int kb = step * KG + group;
        wait_vmcnt_lgkm0<(SLOTS - 2) * kDma>();  // this step has landed, the last one's reads are done
        block_barrier();
        load(step + SLOTS - 1, slot == 0 ? SLOTS - 1 : slot - 1);
        const char* s = smem + slot * kSlot;
        const int shift = 8 * (kb & 3);
        const uint32_t keep = kb < blocks ? 0xFFu : 0u;
        const bool upper = kb * kFp8Block + 64 < K;
        i32x8 x[RM], w[CN];
        uint32_t sx[RM];
        auto frag = [&](const char* p, int off, bool both) {
            const i32x4 lo = lds_read<i32x4>(p, off + 16 * (q ^ sw));
            const i32x4 hi = lds_read<i32x4>(p, off + 16 * ((4 + q) ^ sw));
            return __builtin_shufflevector(lo, both ? hi : i32x4{}, 0, 1, 2, 3, 4, 5, 6, 7);
        };
#pragma unroll
        for (int j = 0; j < CN; ++j) w[j] = frag(s, offW + j * 16 * 128, upper);
        if constexpr (kStepW) ws = lds_read<uint32_t>(s, group * kGroup + kX + kW + 3 * 256);
        if constexpr (QUANT) {
            const bool in = kb * kFp8Block + 8 * r < K;  // channels past K count as zeros
#pragma unroll
            for (int j = 0; j < kDmaX; ++j) {
                const int row = qrow + 16 * j;
                u32x4 v = lds_read<u32x4>(s, group * kGroup + row * 256 + 16 * r);
                if (!in) v = u32x4{0, 0, 0, 0};
                const uint32_t byte = fp8_scale_byte(row16_max(fp8_amax8(v)));
                const float div = fp8_divisor(byte);
                *reinterpret_cast<u32x2*>(xq + row * 128 + 16 * ((r >> 1) ^ fp8_swz(row)) +
                                          8 * (r & 1)) =
                    u32x2{fp8_pack4(v[0], v[1], div), fp8_pack4(v[2], v[3], div)};
                if (r == 0) xs[row] = uint8_t(byte);
            }
            wait_lgkm0();
            block_barrier();
        }
#pragma unroll
        for (int i = 0; i < RM; ++i) x[i] = frag(QUANT ? xq : s, offX + i * 16 * 128, true);
#pragma unroll
        for (int i = 0; i < RM; ++i) {
            if constexpr (QUANT) sx[i] = xs[wm * 16 * RM + 16 * i + r] & keep;
            else sx[i] = (lds_read<uint32_t>(s, offS + i * 64) >> shift) & keep;
        }
        const uint32_t sws = (ws >> shift) & keep;
#pragma unroll
        for (int i = 0; i < RM; ++i)
#pragma unroll
            for (int j = 0; j < CN; ++j)
                acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                    w[j], x[i], acc[i][j], 0, 0, 0, int(sws), 0, int(sx[i]));
        if constexpr (!kStepW) ws = wsp[min((kb + KG) >> 2, words - 1)];
        slot = slot == SLOTS - 1 ? 0 : slot + 1;
    }
    wait_vmcnt_lgkm0<0>();  // the loads past the last step write LDS too
    block_barrier();
    if constexpr (KG > 1) {
        f32x4* join = reinterpret_cast<f32x4*>(smem);
        if (group > 0) {
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
                for (int j = 0; j < CN; ++j)
                    join[(((group - 1) * 4 + wave) * RM * CN + i * CN + j) * 64 + lane] = acc[i][j];
        }
        __syncthreads();
        if (group > 0) return;
#pragma unroll
        for (int g = 0; g < KG - 1; ++g)
#pragma unroll
            for (int i = 0; i < RM; ++i)
#pragma unroll
                for (int j = 0; j < CN; ++j)
                    acc[i][j] += join[((g * 4 + wave) * RM * CN + i * CN + j) * 64 + lane];
    }
#pragma unroll
    for (int i = 0; i < RM; ++i) {
        const int m = row0 + 16 * i + r;
        if (m >= M) continue;
        uint16_t* y = Y + size_t(m) * size_t(N);
#pragma unroll
        for (int j = 0; j < CN; ++j) {
            const int n = col0 + 16 * j + 4 * q;
            const f32x4& v = acc[i][j];
            if (n + 4 <= N) {
                const u32x2 w = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                __builtin_memcpy(y + n, &w, 8);  // one store, at any even address
            } else {
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    if (n + e < N)
                        y[n + e] = __builtin_bit_cast(uint16_t, static_cast<__bf16>(v[e]));
            }
        }
    }
}

template <int RM, int CN, int KG, int SLOTS, bool QUANT = false>
lynx_status launch_mid(const void* X, const uint8_t* Xs, const uint8_t* Wq, const uint8_t* Ws,
                       uint16_t* Y, int M, int N, int K, hipStream_t stream) {
    const int64_t tiles = fp8_tiles(M, N, 32 * RM, 32 * CN);
    hipLaunchKernelGGL((gemm_fp8_mid<RM, CN, KG, SLOTS, QUANT>), dim3(unsigned(tiles)),
                       dim3(256 * KG), 0, stream, X, Xs, Wq, reinterpret_cast<const uint32_t*>(Ws), Y, M, N, K);
    return launch_status();
}

}  // namespace

lynx_status launch_gemm_fp8_mid_quant(const uint16_t* X, const uint8_t* Wq, const uint8_t* Ws,
                                      uint16_t* Y, int M, int N, int K, Fp8Fuse how,
                                      hipStream_t stream) {
    // the tiles and groups of launch_gemm_fp8_mid, two slots of the larger steps
    return how == Fp8Fuse::mid32
               ? launch_mid<1, 1, 4, 2, true>(X, nullptr, Wq, Ws, Y, M, N, K, stream)
               : launch_mid<1, 2, 2, 2, true>(X, nullptr, Wq, Ws, Y, M, N, K, stream);
}

lynx_status launch_gemm_fp8_mid(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                                const uint8_t* Ws, uint16_t* Y, int M, int N, int K, int cus,
                                bool* taken, hipStream_t stream) {
    // The smallest tile of which a compute unit gets no more than one: a second round costs
    // a whole tile's time, and a larger tile leaves units idle.  K = 3072, us: 200 x 3072
    // 64x64 8.4, 32x64 10.6, 96x64 9.8; 333 x 3072 96x64 9.9, 128x64 11.7; 160 x 9216
    // 64x128 12.3, 64x64 15.9, 96x128 14.7; 200 x 9216 96x128 14.9, 128x128 17.2.
    // 128x128 tiles pay against the tiled kernel's where K is long (1024 x 3072 18.0 and
    // 19.7, but K = 1024, N = 4096 9.7 and 8.7), four groups instead of two too (160 x
    // 12288 -> 3072 18.1 and 21.2; K = 1472, N = 1102 5.5 and 5.3; where many rows are
    // quantised inside the product that has two).  Past that the tiled kernel, but for
    // few rows (32 x 73728 32x64 34.8, tiled 45.9; 64 x 73728 64x128 42.4, 46.3) and
    // where only two 64x128 tiles a unit come out even (192 x 18432 20.5, 23.7).
    auto tiles = [&](int tm, int tn) { return fp8_tiles(M, N, tm, tn); };
    auto go = [&](auto kernel) { return kernel(Xq, Xs, Wq, Ws, Y, M, N, K, stream); };
    *taken = true;
    if (tiles(32, 32) <= cus) return go(launch_mid<1, 1, 4, 3>);
    if (tiles(32, 64) <= cus)
        return K >= 4096 && M < 2048 ? go(launch_mid<1, 2, 4, 3>) : go(launch_mid<1, 2, 2, 3>);
    if (tiles(64, 64) <= cus) return go(launch_mid<2, 2, 2, 3>);
    if (tiles(96, 64) <= cus) return go(launch_mid<3, 2, 2, 3>);
    if (tiles(128, 64) <= cus) return go(launch_mid<4, 2, 2, 3>);
    if (tiles(64, 128) <= cus) return go(launch_mid<2, 4, 2, 3>);
    if (tiles(96, 128) <= cus) return go(launch_mid<3, 4, 2, 2>);
    if (tiles(128, 128) <= cus && K > 2048) return go(launch_mid<4, 4, 2, 2>);
    if (M <= 32) return go(launch_mid<1, 2, 2, 3>);
    if (M <= 64 || (tiles(128, 128) > cus && tiles(64, 128) <= 2 * cus))
        return go(launch_mid<2, 4, 1, 3>);
    *taken = false;
    return LYNX_OK;
}

}  // namespace lynx
