// Tiled 8-bit GEMM: Y = sum over K blocks of 2^(ex + ew) (Xq Wq^T), e4m3
// operands with E8M0 block scales, bf16 out (lynx.h).  The instruction and its
// rounding are described in k_gemm_fp8_few.hip; v_mfma_scale_f32_16x16x128_f8f6f4
// is used here too: under sustained load the board's power sets the clock, and a
// loop of this instruction alone reaches 3870 TFLOP/s, of the 32x32x64 one (the
// accumulator read and written for every 64 channels) 3620.
//
// Persistent workgroups of 4 waves walk tiles of 64 NA x 64 NB, each wave
// 32 NA x 32 NB of it as NI x NJ = 2 NA x 2 NB accumulators of 16 x 16 (matrix
// operand A = W, B = X, so that a lane holds runs of a row of Y).  LDS has two slots
// for a K block of X and two for one of W: 128-byte rows (swizzled; whole cache
// lines, so that a line is asked for once) and the X rows' scale words, moved there
// by DMA.
//
// A block is NI NJ instructions, W's fragments one after another against all of X's.
// X's fragments of block p + 1 are read into registers during block p (two sets), W's
// two ahead of their use (a ring of kRing).  So block p reads X's slot p + 1 and W's
// slot p, and there are two barriers to a block:
//   B0 near its start: X of block p + 1 has landed;
//   B1 before its last two W fragments, which have been read: W of block p + 1 has
//      landed; W's slot p is free and takes block p + 2, and X's slot p + 1, whose
//      fragments are all in registers, takes block p + 3 in the next block.
// A slot's loads have about a block's time (2048 cycles at NA = NB = 4) to land, so they
// are issued early, W's right after B1, but X's spread over the block: more of them at
// once hold up the wave that issues them.  9216 x 12288 -> 3072 256 us; with half of W's
// after the next block's start 264.
//
// The blocks run on across tiles: a tile's last two blocks load the next tile's
// first two, in flight during the epilogue.  256 x 256 tiles (the loop for
// an odd number of blocks would spill there: 17% at K = 1152, where a block more costs
// 11) and K <= 128 are filled up to an even number of blocks, and a last block of 64
// channels to 128, with channels loaded again, under scales of 2^-127 for both
// operands, whose products are zero in fp32.
//
// Scales: the scale of row r = l % 16 and the instruction's channels 32 q .. 32 q + 31
// comes from lane l = 16 q + r (a lane's own channels are chunks q and 4 + q of 16).
// X's is the byte of the K block in the row's word (4 blocks); a 16-row piece of W
// lies in one 128-row scale block, so its scale is uniform and comes through the
// scalar cache.
#include <type_traits>
#include <utility>

#include "lynx_fp8.h"
#include "lynx_tile.h"

namespace lynx {
namespace {

// Instructions from .. to - 1 of a block after which no W fragment is read
constexpr int spare(int NI, int from, int to) {
    int n = 0;
    for (int k = from; k < to; ++k) n += k % NI != 2 && k % NI != 3;
    return n;
}

// f(0), ..., f(N - 1) with compile-time arguments
template <typename F, int... I>
__device__ __forceinline__ void for_each(F&& f, std::integer_sequence<int, I...>) {
    (f(std::integral_constant<int, I>{}), ...);
}

// Bytes a wave's epilogue turns at a time: 32 rows of 64 columns, or of 32 where the
// column count or the LDS (shared by two workgroups) does not allow it
constexpr int epilogue_columns(int NA, int NB) { return NA == 4 && NB % 2 == 0 ? 64 : 32; }

// Epilogue of one wave: 32 rows at a time are rounded, turned through the
// wave's own LDS (`ep`) and stored as pieces of rows, 16 bytes a lane: 64 columns
// are full 128-byte lines.  Lane l, r = l % 16, q = l / 16, holds of accumulator (i, j)
// row 16 i + r, columns 16 j + 4 q .. + 3.  16-byte chunks are swizzled by the row, so
// that neither side has bank conflicts.  Rows past M and columns past N are sent past
// the end of the buffer, which drops them; every call issues at least 2 NA NB stores.
// VEC: N % 8 == 0.  Else rows begin at any even address (memory takes such stores), and
// the pieces that N cuts are kept in LDS and stored value by value at the end (from the
// accumulators, or in between, the branches cost 28-51 spilled registers).
template <int NA, int NB, bool VEC>
__device__ __forceinline__ void store_block_rows(const f32x4 (&acc)[2 * NA][2 * NB],
                                                 __amdgpu_buffer_rsrc_t rsY, int N, int row0,
                                                 int col0, char* ep) {
    constexpr int kCols = epilogue_columns(NA, NB);
    constexpr int kChunks = kCols / 8, kPitch = 2 * kCols, kRows = 64 / kChunks;
    constexpr int kCut = 32 * kPitch;
    const int l = fresh_lane();
    const int r = l & 15, q = l >> 4;
    auto swz = [](int row) { return kCols == 64 ? row & 7 : (row >> 1) & 3; };
    const int orow = l / kChunks, och = l % kChunks;
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int c = 0; c < 32 * NB / kCols; ++c) {
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int j = 0; j < kCols / 16; ++j) {
                    const f32x4& v = acc[2 * a + i][c * (kCols / 16) + j];
                    const int row = 16 * i + r;
                    *reinterpret_cast<u32x2*>(ep + row * kPitch +
                                              16 * ((2 * j + (q >> 1)) ^ swz(row)) + 8 * (q & 1)) =
                        u32x2{pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3])};
                }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            const int col = col0 + kCols * c + 8 * och;
#pragma unroll
            for (int i = 0; i < 32 / kRows; ++i) {
                const int lr = i * kRows + orow;
                const int at = lr * kPitch + 16 * (och ^ swz(lr));
                const uint32_t o =
                    (uint32_t(row0 + 32 * a + lr) * uint32_t(N) + uint32_t(col)) * 2u;
                const bool whole = col + 8 <= N;
                const u32x4 w = lds_read<u32x4>(ep, at);
                __builtin_amdgcn_raw_buffer_store_b128(w, rsY, whole ? o : 0xFFFFFFF0u, 0, 0);
                if constexpr (!VEC)  // the others' go to a place that is not read
                    *reinterpret_cast<u32x4*>(
                        ep + kCut + 16 * (!whole && col < N ? 32 * a + lr : 32 * NA)) = w;
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
    if constexpr (!VEC) {
        const int cut = N & ~7;
        if (cut < col0 || cut >= col0 + 32 * NB) return;
#pragma unroll 1
        for (int row = l; row < 32 * NA; row += 64)
#pragma unroll 1
            for (int e = 0; e < N - cut; ++e)
                __builtin_amdgcn_raw_buffer_store_b16(
                    lds_read<uint16_t>(ep, kCut + 16 * row + 2 * e), rsY,
                    (uint32_t(row0 + row) * uint32_t(N) + uint32_t(cut + e)) * 2u, 0, 0);
    }
}

// VEC: N % 8 == 0; ODD: a tile has an odd number of blocks, at least 3 (else an even
// number).  Kernels of their own rather than branches, into whose arms the compiler
// would move the instructions of the block before.
template <int NA, int NB, bool VEC, bool ODD>
__global__ __launch_bounds__(NT, NA == 4 ? 1 : 2) void gemm_fp8_tiled(
    const uint8_t* __restrict__ Xq, const uint8_t* __restrict__ Xs,
    const uint8_t* __restrict__ Wq, const uint32_t* __restrict__ Ws, uint16_t* __restrict__ Y,
    int M, int N, int K) {
    constexpr int TM = 64 * NA, TN = 64 * NB;
    constexpr int NI = 2 * NA, NJ = 2 * NB;         // accumulators per wave
    constexpr int kRow = 128;                       // LDS bytes per row and block
    constexpr int kX = TM * kRow + 1024;            // a slot of X: + a scale word per row (256 places)
    constexpr int kW = TN * kRow;                   // a slot of W
    constexpr int kDmaX = 2 * NA + 1, kDmaW = 2 * NB;  // DMA instructions per wave and block
    constexpr int kRing = NB == 3 ? 3 : 4;          // W fragments in registers; divides NJ
    constexpr int kM = NI * NJ;                     // matrix instructions per wave and block
    // The barriers follow these instructions
    constexpr int kB0 = NA == 2 ? 1 : NB == 3 ? 8 : 12, kB1 = (NJ - 2) * NI + 1;
    constexpr int kRead = (NJ - 3) * NI + 1;        // X is read before this one
    // X's loads are issued from this one (ODD: after B0, for the fragments that are read
    // again at a tile's end) ...
    constexpr int kFromX = ODD ? kB0 : NA == 2 ? 0 : 5;
    constexpr int kEndX = NA == 2 ? kB1 : NB == 3 ? 32 : 48;  // ... and before this one
    constexpr int kEarlyX = spare(NI, kFromX, kB0) * kDmaX / spare(NI, kFromX, kEndX);  // before B0
    constexpr int kStores = 2 * NA * NB;            // stores of an epilogue, at least
    // a wave's LDS for the epilogue
    constexpr int kEp = 64 * epilogue_columns(NA, NB) + (VEC ? 0 : 16 * (32 * NA + 1));
    constexpr int kBS = NB == 3 ? NB : 1;           // scale blocks a wave's columns touch
    // rows of tiles that an XCD walks down together.  16384 x 4096 -> 4096 6 rows 201 us, 4
    // 208, 8 217; 9216 x 3072 -> 12288 270, 266, 274; 256 x 192 tiles, 6000 x 4096 -> 11008
    // 234, 221, 228.  Eight rows of 128 for the small tiles, two workgroups a unit.
    constexpr int kGroup = NA == 2 ? 8 : NB == 3 ? 4 : 6;
    // past the end of X and W (they hold less than 2^31 bytes, and a tile's rows
    // span less than 2^31: kPast plus a row's offset does not wrap)
    constexpr uint32_t kPast = 0x80000000u;
    constexpr int kOffW = 2 * kX, kOffEp = 2 * kX + 2 * kW, kLds = kOffEp + 4 * kEp;
    static_assert(NJ % kRing == 0 && kEndX <= kB1 && kB0 < kRead, "schedule");
    static_assert(kLds <= 160 * 1024 / (NA == 4 ? 1 : 2), "LDS budget");
    static_assert(kStores + kDmaX < 64 && kStores + kDmaW + kEarlyX < 64, "vmcnt range");
    __shared__ __attribute__((aligned(1024))) char smem[kLds];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int r = lane & 15, q = lane >> 4;
    const int wm = wave & 1, wn = wave >> 1;
    const int tiles_m = (M + TM - 1) / TM, tiles_n = (N + TN - 1) / TN;
    const int ntiles = tiles_m * tiles_n;
    const int real = (K + 127) / 128;               // blocks that hold channels of K
    const int np = ODD ? real : (real + 1) & ~1;    // blocks of a tile
    const int words = fp8_scale_words(K);
    const int nblocks = (N + kFp8Block - 1) / kFp8Block;

    // ---- loads: DMA instruction j of wave w moves rows 8 w + l/8 + 32 j of an
    // operand, lane l's 16 bytes the chunk that the row's swizzle puts there (the
    // same chunk for every j)
    const uint32_t lds0 = lds_addr(smem);
    const i32x4 rsX = make_rsrc(Xq, uint32_t(M) * uint32_t(K));
    const i32x4 rsW = make_rsrc(Wq, uint32_t(N) * uint32_t(K));
    const i32x4 rsS = make_rsrc(Xs, uint32_t(words) * uint32_t(M) * 4u);
    const int chunk = (lane & 7) ^ fp8_swz(8 * wave + (lane >> 3));
    struct Aim {
        uint32_t x, w, s;  // a tile's offsets, of instruction j = 0
    };
    // Past the last tile the loads go on, so that every wait has the same count, but
    // from past the ends of the buffers: they read nothing.
    auto aim = [&](int v) {
        int tm, tn;
        tile_of(min(v, ntiles - 1), tiles_m, tiles_n, tm, tn, kGroup);
        const bool past = v >= ntiles;
        const int l = fresh_lane();
        const uint32_t row = uint32_t(8 * wave + (l >> 3)), c = uint32_t(16 * chunk);
        const uint32_t x = (uint32_t(tm * TM) + row) * uint32_t(K) + c;
        const uint32_t w = (uint32_t(tn * TN) + row) * uint32_t(K) + c;
        // the word's offset goes into the scalar part, which is not range checked:
        // rows past the end take the last row's words
        const uint32_t s = uint32_t(min(tm * TM + 64 * (wave % NA) + l, M - 1)) * 4u;
        return Aim{past ? kPast : x, past ? kPast : w, past ? kPast : s};
    };
    // Where a block has only 64 channels, the upper chunks load the lower ones again;
    // a block past the last loads the last again.
    auto back_of = [&](int p) { return p * kRow + 64 < K || chunk < 4 ? 0u : 64u; };
    auto dma_x = [&](int slot, uint32_t x, uint32_t s, int p, int i) {
        const uint32_t base = lds0 + uint32_t(slot);
        const int pr = min(p, real - 1);
        if (i < kDmaX - 1)
            dma16(base + 1024 * (wave + 4 * i), x - back_of(pr) + uint32_t(32 * i) * uint32_t(K), rsX,
                  uint32_t(pr * kRow));
        else
            dma4(base + TM * kRow + 256 * wave, s, rsS, uint32_t(pr >> 2) * uint32_t(M) * 4u);
    };
    auto dma_w = [&](int slot, uint32_t w, int p, int i) {
        const int pr = min(p, real - 1);
        dma16(lds0 + kOffW + uint32_t(slot) + 1024 * (wave + 4 * i),
              w - back_of(pr) + uint32_t(32 * i) * uint32_t(K), rsW, uint32_t(pr * kRow));
    };

    // ---- fragments and instructions
    const int swz = fp8_swz(r);
    const int offX = (wm * 32 * NA + r) * kRow, offS = TM * kRow + (wm * 32 * NA + r) * 4;
    const int offW = kOffW + (wn * 32 * NB + r) * kRow;
    struct Frag {
        i32x4 lo, hi;
    };
    Frag x[2][NI], w[kRing];
    uint32_t sx[NI], sw[kBS];       // scale words of the block at hand
    uint32_t sxn[NI], swn[kBS];     // and of the next
    const uint32_t* wsp[kBS];       // the tile's scale words of W
    auto read = [&](int off, Frag& f, int part) {
        (part ? f.hi : f.lo) = lds_read<i32x4>(smem, off + 16 * ((4 * part + q) ^ swz));
    };
    f32x4 acc[NI][NJ];
    int slot = 0;                   // 0 or 1: of the block at hand
    int lpx = 0, lpw = 0;           // the blocks being loaded
    uint32_t atx = 0, ats = 0, atw = 0;  // and their offsets
    Aim next = {0, 0, 0};           // the next tile's
    // Block p on fragment set S: waits for X (B0) and W (B1) until at most wait0 and
    // wait1 later vector memory operations are under way; issues X's loads, then W's.
    auto block = [&](auto set, auto first, auto wait0, auto wait1, int p) {
        constexpr int S = decltype(set)::value;
        const int oth = 1 - slot;
        const int shift = 8 * (p & 3);                    // the block's byte in the scale words
        // 2^-127 for the channels it is filled up with
        const uint32_t keep = p * kRow + 64 * (q >> 1) < K ? 0xFFu : 0u;
        if (++lpx >= np) lpx = 0;
        const bool over = lpx < 2;  // the next tile's
        atx = over ? next.x : atx;
        ats = over ? next.s : ats;
        for_each([&](auto kc) {
            constexpr int k = decltype(kc)::value, i = k % NI, j = k / NI;
            const Frag &fx = x[S][i], &fw = w[j % kRing];
            const i32x8 vx = __builtin_shufflevector(fx.lo, fx.hi, 0, 1, 2, 3, 4, 5, 6, 7);
            const i32x8 vw = __builtin_shufflevector(fw.lo, fw.hi, 0, 1, 2, 3, 4, 5, 6, 7);
            acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
                vw, vx, decltype(first)::value ? f32x4{} : acc[i][j], 0, 0, 0,
                int((sw[kBS == 1 ? 0 : j / 2] >> shift) & keep), 0, int((sx[i] >> shift) & keep));
            if constexpr (k == kB0) {
                wait_vmcnt_lgkm0<decltype(wait0)::value>();
                block_barrier();
            }
            if constexpr (k == kRead) {
                // A scalar load under way turns every wait for LDS reads into a wait for all
                // of them: it stands after the last read of X, half a dozen instructions
                // before the next wait.
                const int wd = min((p + 1) >> 2, words - 1);
#pragma unroll
                for (int b = 0; b < kBS; ++b) swn[b] = wsp[b][wd];
            }
            if constexpr (k == kB1) {
                wait_vmcnt_lgkm0<decltype(wait1)::value>();
                block_barrier();
            }
            // W's fragment j + 2, of the next block at the end
            constexpr bool w_read = k % NI == 2 || k % NI == 3;
            if constexpr (w_read) {
                constexpr int n = (j + 2) % NJ;
                const int sl = j + 2 < NJ ? slot : oth;
                read(offW + sl * kW + n * 16 * kRow, w[(j + 2) % kRing], k % NI - 2);
            }
            // the other memory instructions stand where W is not read: X's fragments and
            // scales (two rows' to an instruction) of the next block ...
            if constexpr (!w_read && k > kB0 && k < kRead) {
                constexpr int g = spare(NI, kB0 + 1, kRead), t = spare(NI, kB0 + 1, k), n = 5 * NI / 2;
                for_each([&](auto mc) {
                    constexpr int m = t * n / g + decltype(mc)::value;
                    if constexpr (m % 5 < 4) {
                        constexpr int f = m / 5 * 4 + m % 5;
                        read(offX + oth * kX + (f / 2) * 16 * kRow, x[1 - S][f / 2], f % 2);
                    } else {
                        constexpr int f = m / 5;
                        sxn[f] = lds_read<uint32_t>(smem, oth * kX + offS + f * 64);
                        sxn[f + NI / 2] = lds_read<uint32_t>(smem, oth * kX + offS + (f + NI / 2) * 64);
                    }
                }, std::make_integer_sequence<int, (t + 1) * n / g - t * n / g>{});
            }
            // ... and the loads
            if constexpr (!w_read && k >= kFromX && k < kEndX) {
                constexpr int g = spare(NI, kFromX, kEndX), t = spare(NI, kFromX, k);
#pragma unroll
                for (int n = t * kDmaX / g; n < (t + 1) * kDmaX / g; ++n)
                    dma_x(slot * kX, atx, ats, lpx, n);
            }
            if constexpr (k == kB1) {
                lpw = lpx;
                atw = over ? next.w : atw;
            }
            if constexpr (!w_read && k > kB1) {
                constexpr int g = spare(NI, kB1 + 1, kM), t = spare(NI, kB1 + 1, k);
#pragma unroll
                for (int n = t * kDmaW / g; n < (t + 1) * kDmaW / g; ++n)
                    dma_w(slot * kW, atw, lpw, n);
            }
            __builtin_amdgcn_sched_barrier(0);
        }, std::make_integer_sequence<int, kM>{});
        slot = oth;
#pragma unroll
        for (int i = 0; i < NI; ++i) sx[i] = sxn[i];
#pragma unroll
        for (int b = 0; b < kBS; ++b) sw[b] = swn[b];
    };

    const __amdgpu_buffer_rsrc_t rsY =
        __builtin_amdgcn_make_buffer_rsrc(Y, 0, int(uint32_t(M) * uint32_t(N) * 2u), kRsrcWord3);
    {
        const Aim at = aim(blockIdx.x);
        atx = at.x;
        ats = at.s;
        atw = at.w;
    }
#pragma unroll
    for (int p = 0; p < 2; ++p) {
#pragma unroll
        for (int i = 0; i < kDmaX; ++i) dma_x(p * kX, atx, ats, p, i);
#pragma unroll
        for (int i = 0; i < kDmaW; ++i) dma_w(p * kW, atw, p, i);
    }
    wait_vmcnt<0>();  // both: no stores stand between them and the first waits
    block_barrier();
#pragma unroll
    for (int n = 0; n < 2 * NI; ++n) read(offX + (n / 2) * 16 * kRow, x[0][n / 2], n % 2);
#pragma unroll
    for (int n = 0; n < 4; ++n) read(offW + (n / 2) * 16 * kRow, w[n / 2], n % 2);
#pragma unroll
    for (int i = 0; i < NI; ++i) sx[i] = lds_read<uint32_t>(smem, offS + i * 64);
    wait_lgkm0();
    block_barrier();  // the first block loads into X's slot before its B0

    using S0 = std::integral_constant<int, 0>;
    using S1 = std::integral_constant<int, 1>;
    using First = std::true_type;
    using Other = std::false_type;
    using AfterW = std::integral_constant<int, kDmaW + kEarlyX>;  // and this block's first of X
    using AfterX = std::integral_constant<int, kDmaX>;
    // a tile's first waits pass over the last one's stores: its first two blocks were
    // loaded before them
    using Stores0 = std::integral_constant<int, kDmaW + kEarlyX + kStores>;
    using Stores1 = std::integral_constant<int, kDmaX + kStores>;
    for (int v = blockIdx.x; v < ntiles; v += gridDim.x) {
        int tm, tn;
        tile_of(v, tiles_m, tiles_n, tm, tn, kGroup);
        const int row0 = tm * TM + wm * 32 * NA, col0 = tn * TN + wn * 32 * NB;
#pragma unroll
        for (int b = 0; b < kBS; ++b)
            wsp[b] = Ws + size_t(__builtin_amdgcn_readfirstlane(
                              min((col0 + 32 * b) / kFp8Block, nblocks - 1))) * size_t(words);
#pragma unroll
        for (int b = 0; b < kBS; ++b) sw[b] = wsp[b][0];
        next = aim(v + int(gridDim.x));
        lpx = lpw = 1;  // block p loads block p + 2, or the next tile's p + 2 - np
        block(S0{}, First{}, Stores0{}, Stores1{}, 0);
        if constexpr (ODD) {
            int p = 1;
            do {
                block(S1{}, Other{}, AfterW{}, AfterX{}, p);
                block(S0{}, Other{}, AfterW{}, AfterX{}, p + 1);
                p += 2;
            } while (p < np);
            // the next tile begins with set 0 again: its fragments now that it is free (their
            // slot stays as it is until that tile's B1)
#pragma unroll
            for (int n = 0; n < 2 * NI; ++n)
                read(offX + slot * kX + (n / 2) * 16 * kRow, x[0][n / 2], n % 2);
        } else {
            for (int p = 1; p < np - 2; p += 2) {
                block(S1{}, Other{}, AfterW{}, AfterX{}, p);
                block(S0{}, Other{}, AfterW{}, AfterX{}, p + 1);
            }
            block(S1{}, Other{}, AfterW{}, AfterX{}, np - 1);
        }
        store_block_rows<NA, NB, VEC>(acc, rsY, N, row0, col0, smem + kOffEp + wave * kEp);
    }
    wait_vmcnt<0>();  // the loads past the last tile still write LDS
}

template <int NA, int NB>
lynx_status launch_tiled(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                         const uint8_t* Ws, uint16_t* Y, int M, int N, int K, int cus,
                         hipStream_t stream) {
    const long tiles = long((M + 64 * NA - 1) / (64 * NA)) * ((N + 64 * NB - 1) / (64 * NB));
    const long most = long(cus) * (NA == 4 ? 1 : 2);
    const dim3 grid(unsigned(tiles < most ? tiles : most));
    const uint32_t* ws = reinterpret_cast<const uint32_t*>(Ws);
    auto launch = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, grid, dim3(NT), 0, stream, Xq, Xs, Wq, ws, Y, M, N, K);
    };
    constexpr bool kOdd = !(NA == 4 && NB == 4);
    const bool odd = kOdd && K > 128 && (K + 127) / 128 % 2 != 0;
    if (N % 8 == 0) {
        if (odd) launch(gemm_fp8_tiled<NA, NB, true, kOdd>);
        else launch(gemm_fp8_tiled<NA, NB, true, false>);
    } else {
        if (odd) launch(gemm_fp8_tiled<NA, NB, false, kOdd>);
        else launch(gemm_fp8_tiled<NA, NB, false, false>);
    }
    return launch_status();
}

}  // namespace

lynx_status launch_gemm_fp8(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                            const uint8_t* Ws, uint16_t* Y, int M, int N, int K,
                            hipStream_t stream) {
    if (fp8_is_few(M, N)) return launch_gemm_fp8_few(Xq, Xs, Wq, Ws, Y, M, N, K, stream);
    int cus = 0;
    if (device_cu_count(&cus) != LYNX_OK) return LYNX_ERR_DEVICE;
    bool taken = false;
    const lynx_status st = launch_gemm_fp8_mid(Xq, Xs, Wq, Ws, Y, M, N, K, cus, &taken, stream);
    if (taken) return st;
    // Rounds of tiles over the compute units, each at its tile's time relative to a
    // 256 x 256 one (measured at K = 3072: 33 us; 256 x 192 0.83 of that; 128 x 128, two
    // workgroups a unit, 0.75, 0.45 with at most one).  4096 x 9216: 256 x 192 101 us,
    // 256 x 256 115; 9216 x 3072: 89 and 75; 512 x 12288: 128 x 128 25, 256 x 192 28.
    auto tiles = [&](int tm, int tn) { return fp8_tiles(M, N, tm, tn); };
    auto rounds = [](long t, long n) { return (t + n - 1) / n; };
    const long np = (K + 127) / 128;  // 256 x 256 tiles take an even number of K blocks
    const long wide = rounds(tiles(256, 256), cus) * (100 * ((np + 1) & ~1L) / np);
    const long mid = rounds(tiles(256, 192), cus) * 83;
    const long t22 = tiles(128, 128);
    const long small = t22 <= cus ? 45 : rounds(t22, 2 * cus) * 75;
    if (small < wide && small < mid)
        return launch_tiled<2, 2>(Xq, Xs, Wq, Ws, Y, M, N, K, cus, stream);
    return mid < wide ? launch_tiled<4, 3>(Xq, Xs, Wq, Ws, Y, M, N, K, cus, stream)
                      : launch_tiled<4, 4>(Xq, Xs, Wq, Ws, Y, M, N, K, cus, stream);
}

}  // namespace lynx
