// Tiled 8-bit GEMM: Y = sum over K blocks of 2^(ex + ew) (Xq Wq^T), e4m3
// operands with E8M0 block scales, bf16 out (lynx.h).  The instruction and its
// rounding are described in k_gemm_fp8_few.hip.
//
// Persistent workgroups of 4 waves walk tiles of 64 NA x 64 NB, each wave
// 32 NA x 32 NB of it as NA x NB accumulators of 32 x 32 (matrix operand A = W,
// B = X, so that a lane holds runs of a row of Y).  LDS has two slots of one K
// block each: 128-byte rows of X and W (swizzled; whole cache lines, so that a
// line is asked for once) and the rows' scale words, moved there by DMA.  A block is
// two stages of 64 channels, at NA = NB = 4 16 instructions of 64 cycles a wave
// each.  A stage's fragments are read from LDS into registers during the stage
// before it (two sets, 32 bytes of a row per lane and accumulator row or column).
// So the second stage of block p reads from block p + 1's slot and finds block p's
// slot free: it opens with the block's only barrier, after which block p + 1 has
// landed for all waves, and begins to load block p + 2 into slot p.  The loads are
// spread over the instructions of this stage and the first half of the next: in a
// burst they hold up the wave that issues them (4 instructions' room instead of 22:
// 10% of the time).
//
// The blocks run on across tiles: a tile's last two second stages load the next
// tile's first two blocks, in flight during the epilogue.  A tile has at least two
// blocks; K <= 128, and a last block of 64 channels, are filled up with channels
// loaded again, under scales of 2^-127 for both operands, whose products are zero
// in fp32.
//
// Scales: lane l's B operand is row l % 32 of X, its scale the byte of the K block
// in that row's word (4 blocks); a 32-row piece of W lies in one 128-row scale
// block, so its scale is uniform and comes through the scalar cache.
#include <type_traits>

#include "lynx_fp8.h"
#include "lynx_tile.h"

namespace lynx {
namespace {

typedef uint32_t lds_u32x2 __attribute__((ext_vector_type(2)));

// 32-column blocks that an epilogue turns at a time: 2, or 1 where NB is odd or LDS
// is shared by two workgroups
constexpr int epilogue_blocks(int NA, int NB) { return NA == 4 && NB % 2 == 0 ? 2 : 1; }

// Epilogue of one wave, N % 8 == 0: 32 rows x 32 CB columns at a time are rounded,
// turned through the wave's own LDS (`ep`) and stored as whole rows, 16 bytes a
// lane: CB = 2 writes full 128-byte lines.  Lane l, r = l % 32, h = l / 32, holds of
// accumulator (a, b) row 32 a + r, columns 32 b + 8 (e / 4) + 4 h + e % 4.  16-byte
// chunks are swizzled by the row, so that neither side has bank conflicts.  Rows
// past M and columns past N are sent past the end of the buffer, which drops them;
// every call issues NA NB 2 stores.
template <int NA, int NB>
__device__ __forceinline__ void store_block_rows(const f32x16 (&acc)[NA][NB],
                                                 __amdgpu_buffer_rsrc_t rsY, int N, int row0,
                                                 int col0, char* ep) {
    constexpr int CB = epilogue_blocks(NA, NB);
    constexpr int kChunks = 4 * CB, kPitch = 16 * kChunks, kRows = 64 / kChunks;
    const int l = fresh_lane();
    const int r = l & 31, h = l >> 5;
    auto swz = [](int row) { return CB == 2 ? row & 7 : (row >> 1) & 3; };
    const int orow = l / kChunks, och = l % kChunks;
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int bp = 0; bp < NB / CB; ++bp) {
#pragma unroll
            for (int b = 0; b < CB; ++b)
#pragma unroll
                for (int g = 0; g < 4; ++g) {
                    const f32x16& v = acc[a][bp * CB + b];
                    *reinterpret_cast<lds_u32x2*>(ep + r * kPitch + 16 * ((4 * b + g) ^ swz(r)) +
                                                  8 * h) =
                        lds_u32x2{pack_bf16x2(v[4 * g], v[4 * g + 1]),
                                  pack_bf16x2(v[4 * g + 2], v[4 * g + 3])};
                }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            const int col = col0 + 32 * CB * bp + 8 * och;
#pragma unroll
            for (int i = 0; i < 32 / kRows; ++i) {
                const int lr = i * kRows + orow;
                const u32x4 w = lds_read<u32x4>(ep, lr * kPitch + 16 * (och ^ swz(lr)));
                const uint32_t o =
                    (uint32_t(row0 + 32 * a + lr) * uint32_t(N) + uint32_t(col)) * 2u;
                __builtin_amdgcn_raw_buffer_store_b128(w, rsY, col < N ? o : 0xFFFFFFF0u, 0, 0);
            }
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
        }
}

// Epilogue for other N: every lane stores its values one by one.
template <int NA, int NB>
__device__ __forceinline__ void store_block_single(const f32x16 (&acc)[NA][NB],
                                                   __amdgpu_buffer_rsrc_t rsY, int N, int row0,
                                                   int col0) {
    const int l = fresh_lane();
    const int r = l & 31, h = l >> 5;
#pragma unroll
    for (int a = 0; a < NA; ++a)
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                const int col = col0 + 32 * b + 8 * (e / 4) + 4 * h + e % 4;
                const uint32_t o = (uint32_t(row0 + 32 * a + r) * uint32_t(N) + uint32_t(col)) * 2u;
                __builtin_amdgcn_raw_buffer_store_b16(
                    __builtin_bit_cast(uint16_t, static_cast<__bf16>(acc[a][b][e])), rsY,
                    col < N ? o : 0xFFFFFFF0u, 0, 0);
            }
}

// VEC: N % 8 == 0 (two kernels rather than a branch before the epilogue, into whose
// arms the compiler would move the last stage's instructions)
template <int NA, int NB, bool VEC>
__global__ __launch_bounds__(NT, NA == 4 ? 1 : 2) void gemm_fp8_tiled(
    const uint8_t* __restrict__ Xq, const uint8_t* __restrict__ Xs,
    const uint8_t* __restrict__ Wq, const uint32_t* __restrict__ Ws, uint16_t* __restrict__ Y,
    int M, int N, int K) {
    constexpr int TM = 64 * NA, TN = 64 * NB;
    constexpr int kRow = 128;                       // LDS bytes per row and block
    constexpr int kX = TM * kRow, kW = TN * kRow;
    constexpr int kSlot = kX + kW + 1024;           // + a scale word per row (256 places)
    constexpr int kDmaX = 2 * NA, kDmaW = 2 * NB;   // DMA instructions per wave and block
    constexpr int kDma = kDmaX + kDmaW + 1;
    constexpr int kM = NA * NB;                     // matrix instructions per wave and stage
    constexpr int kReads = 2 * (NA + NB);           // 16-byte LDS reads per wave and stage
    constexpr int kBar = kM >= 12 ? 1 : 0;          // the barrier follows instruction kBar
    constexpr int kTail = kM / 8;                   // instructions after the last LDS read
    constexpr int kLoad1 = kDma * 3 / 5;            // loads issued in a block's second stage,
    constexpr int kGaps0 = kM / 2;                  // the others here, early in the next
    constexpr int kStores = 2 * NA * NB;            // stores of an epilogue, at least
    constexpr int kEp = 2048 * epilogue_blocks(NA, NB);  // a wave's LDS for the epilogue
    constexpr int kBS = NB == 3 ? NB : 1;           // scale blocks a wave's columns touch
    // past the end of X and W (they hold less than 2^31 bytes, and a tile's rows
    // span less than 2^31: kPast plus a row's offset does not wrap)
    constexpr uint32_t kPast = 0x80000000u;
    static_assert(2 * kSlot + 4 * kEp <= 160 * 1024 / (NA == 4 ? 1 : 2), "LDS budget");
    static_assert(kStores < 64, "vmcnt range");
    __shared__ __attribute__((aligned(1024))) char smem[2 * kSlot + 4 * kEp];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int r = lane & 31, h = lane >> 5;
    const int wm = wave & 1, wn = wave >> 1;
    const int tiles_m = (M + TM - 1) / TM, tiles_n = (N + TN - 1) / TN;
    const int ntiles = tiles_m * tiles_n;
    const int real = K / 64;                        // stages that hold channels of K
    const int np = max((real + 1) / 2, 2);          // blocks of a tile
    const int words = fp8_scale_words(K);
    const int nblocks = (N + kFp8Block - 1) / kFp8Block;

    // ---- loads: DMA instruction j of wave w moves rows 8 w + l/8 + 32 j of an
    // operand, lane l's 16 bytes the chunk that the row's swizzle puts there (the
    // same chunk for every j)
    const uint32_t lds0 = lds_addr(smem);
    const i32x4 rsX = make_rsrc(Xq, uint32_t(M) * uint32_t(K));
    const i32x4 rsW = make_rsrc(Wq, uint32_t(N) * uint32_t(K));
    const i32x4 rsS = make_rsrc(Xs, uint32_t(words) * uint32_t(M) * 4u);
    const int chunk = (lane & 7) ^ swz128(8 * wave + (lane >> 3));
    struct Aim {
        uint32_t x, w, s;  // a tile's offsets, of instruction j = 0
    };
    // Past the last tile the loads go on, so that every wait has the same count, but
    // from past the ends of the buffers: they read nothing.
    auto aim = [&](int v) {
        int tm, tn;
        tile_of(min(v, ntiles - 1), tiles_m, tiles_n, tm, tn);
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
    // DMA instruction i of block p.  Where the block has only 64 channels, the upper
    // chunks load the lower ones again; a block past the last loads the last again.
    auto dma = [&](int slot, const Aim& t, int p, int i) {
        const uint32_t base = lds0 + uint32_t(slot);
        const int pr = min(p, (real - 1) >> 1);
        const uint32_t back = 2 * pr + 1 < real || chunk < 4 ? 0u : 64u;
        if (i < kDmaX)
            dma16(base + 1024 * (wave + 4 * i), t.x - back + uint32_t(32 * i) * uint32_t(K), rsX,
                  uint32_t(pr * kRow));
        else if (i < kDmaX + kDmaW)
            dma16(base + kX + 1024 * (wave + 4 * (i - kDmaX)),
                  t.w - back + uint32_t(32 * (i - kDmaX)) * uint32_t(K), rsW, uint32_t(pr * kRow));
        else
            dma4(base + kX + kW + 256 * wave, t.s, rsS, uint32_t(pr >> 2) * uint32_t(M) * 4u);
    };

    // ---- fragments and instructions
    const int s128 = swz128(r);
    const int offX = (wm * 32 * NA + r) * kRow, offW = kX + (wn * 32 * NB + r) * kRow;
    const int offS = kX + kW + (wm * 32 * NA + r) * 4;
    struct Frags {
        i32x4 x[NA][2], w[NB][2];
    };
    Frags fr[2];
    uint32_t sx[NA], sw[kBS];       // scale words of the block at hand
    uint32_t sxn[NA], swn[kBS];     // and of the next
    const uint32_t* wsp[kBS];       // the tile's scale words of W
    auto read_n = [&](int slot, int half, Frags& f, int n) {
        const int blk = n >> 1, part = n & 1;
        const int c = 16 * ((4 * half + 2 * part + h) ^ s128);
        if (blk < NA)
            f.x[blk][part] = lds_read<i32x4>(smem + slot, offX + blk * 32 * kRow + c);
        else
            f.w[blk - NA][part] = lds_read<i32x4>(smem + slot, offW + (blk - NA) * 32 * kRow + c);
    };
    auto read_scales = [&](int slot, uint32_t* s) {
#pragma unroll
        for (int a = 0; a < NA; ++a) s[a] = lds_read<uint32_t>(smem + slot, offS + a * 128);
    };
    f32x16 acc[NA][NB];
    auto mma = [&](const Frags& f, int k, int shift, uint32_t keep, auto first) {
        const int a = k % NA, b = k / NA;
        const i32x8 vx = __builtin_shufflevector(f.x[a][0], f.x[a][1], 0, 1, 2, 3, 4, 5, 6, 7);
        const i32x8 vw = __builtin_shufflevector(f.w[b][0], f.w[b][1], 0, 1, 2, 3, 4, 5, 6, 7);
        acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            vw, vx, decltype(first)::value ? f32x16{} : acc[a][b], 0, 0, 0,
            int((sw[kBS == 1 ? 0 : b] >> shift) & keep), 0, int((sx[a] >> shift) & keep));
    };
    int cur = 0;  // slot of the block at hand
    // Stage `half` of block p on fragment set `half`: its instructions and the next
    // stage's LDS reads.  A second half waits until at most `wait` later vector
    // memory operations are under way, reads the next block's scale words and issues
    // the first `loads` loads of block lp (aimed at `t`) into the slot it frees; a
    // first half issues the others of the block that the stage before began.
    auto stage = [&](auto half, auto first, auto wait, auto loads, int p, const Aim& t, int lp) {
        constexpr int S = decltype(half)::value, kLoads = decltype(loads)::value;
        constexpr int kB0 = S == 1 ? kBar + 1 : 0;        // the first read's place
        constexpr int kReadIn = kM - kTail - kB0, kLoadIn = S == 1 ? kM - kB0 : kGaps0;
        constexpr int kFrom = S == 1 ? 0 : kDma - kLoads;
        const int nxt = S == 1 ? kSlot - cur : cur;       // where the reads go
        const int shift = 8 * (p & 3);                    // the block's byte in the scale words
        const uint32_t keep = 2 * p + S < real ? 0xFFu : 0u;  // 2^-127 where filled up
#pragma unroll
        for (int k = 0; k < kM; ++k) {
            mma(fr[S], k, shift, keep, first);
            if (S == 0 && k == 0) {
                // here, so that the scalar load has a stage's time before a wait counts it
                const int w = min((p + 1) >> 2, words - 1);
#pragma unroll
                for (int b = 0; b < kBS; ++b) swn[b] = wsp[b][w];
            }
            if (S == 1 && k == kBar) {
                wait_vmcnt_lgkm0<decltype(wait)::value>();
                block_barrier();
                read_scales(nxt, sxn);
            }
            const int q = k - kB0;
            if (q >= 0 && q < kLoadIn) {
#pragma unroll
                for (int i = q * kLoads / kLoadIn; i < (q + 1) * kLoads / kLoadIn; ++i)
                    dma(S == 1 ? cur : kSlot - cur, t, lp, kFrom + i);
            }
            if (q >= 0 && q < kReadIn) {
#pragma unroll
                for (int n = q * kReads / kReadIn; n < (q + 1) * kReads / kReadIn; ++n)
                    read_n(nxt, 1 - S, fr[1 - S], n);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        if (S == 1) {
            cur = nxt;
#pragma unroll
            for (int a = 0; a < NA; ++a) sx[a] = sxn[a];
#pragma unroll
            for (int b = 0; b < kBS; ++b) sw[b] = swn[b];
        }
    };

    const __amdgpu_buffer_rsrc_t rsY =
        __builtin_amdgcn_make_buffer_rsrc(Y, 0, int(uint32_t(M) * uint32_t(N) * 2u), kRsrcWord3);
    Aim at = aim(blockIdx.x);
#pragma unroll
    for (int p = 0; p < 2; ++p)
#pragma unroll
        for (int i = 0; i < kDma; ++i) dma(p * kSlot, at, p, i);
    wait_vmcnt<0>();  // both: no stores stand between them and the first wait
    block_barrier();
    read_scales(0, sx);
#pragma unroll
    for (int n = 0; n < kReads; ++n) read_n(0, 0, fr[0], n);

    using H0 = std::integral_constant<int, 0>;
    using H1 = std::integral_constant<int, 1>;
    using None = std::integral_constant<int, 0>;
    using Some = std::integral_constant<int, kLoad1>;
    using Rest = std::integral_constant<int, kDma - kLoad1>;
    using All = std::integral_constant<int, kDma>;
    using Stores = std::integral_constant<int, kStores>;
    for (int v = blockIdx.x; v < ntiles; v += gridDim.x) {
        int tm, tn;
        tile_of(v, tiles_m, tiles_n, tm, tn);
        const int row0 = tm * TM + wm * 32 * NA, col0 = tn * TN + wn * 32 * NB;
#pragma unroll
        for (int b = 0; b < kBS; ++b)
            wsp[b] = Ws + size_t(__builtin_amdgcn_readfirstlane(
                              min((col0 + 32 * b) / kFp8Block, nblocks - 1))) * size_t(words);
#pragma unroll
        for (int b = 0; b < kBS; ++b) sw[b] = wsp[b][0];
        const Aim next = aim(v + int(gridDim.x));
        // block p's second stage loads block p + 2, or the next tile's p + 2 - np
        int lp = 2;
        auto cross = [&] {
            if (lp >= np) lp -= np;
            const bool over = lp < 2;
            at = Aim{over ? next.x : at.x, over ? next.w : at.w, over ? next.s : at.s};
        };
        stage(H0{}, std::true_type{}, None{}, None{}, 0, at, 0);
        cross();
        // the first wait of a tile passes over the last one's stores: block 1 was
        // loaded before them
        stage(H1{}, std::false_type{}, Stores{}, Some{}, 0, at, lp);
        for (int p = 1; p < np - 1; ++p) {
            stage(H0{}, std::false_type{}, None{}, Rest{}, p, at, lp);
            ++lp;
            cross();
            stage(H1{}, std::false_type{}, None{}, Some{}, p, at, lp);
        }
        stage(H0{}, std::false_type{}, None{}, Rest{}, np - 1, at, lp);
        stage(H1{}, std::false_type{}, None{}, All{}, np - 1, at, 1);
        if constexpr (VEC)
            store_block_rows(acc, rsY, N, row0, col0, smem + 2 * kSlot + wave * kEp);
        else
            store_block_single(acc, rsY, N, row0, col0);
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
    if (N % 8 == 0)
        hipLaunchKernelGGL((gemm_fp8_tiled<NA, NB, true>), grid, dim3(NT), 0, stream, Xq, Xs, Wq,
                           ws, Y, M, N, K);
    else
        hipLaunchKernelGGL((gemm_fp8_tiled<NA, NB, false>), grid, dim3(NT), 0, stream, Xq, Xs, Wq,
                           ws, Y, M, N, K);
    return launch_status();
}

}  // namespace

lynx_status launch_gemm_fp8(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                            const uint8_t* Ws, uint16_t* Y, int M, int N, int K,
                            hipStream_t stream) {
    if (M <= kFewRows) return launch_gemm_fp8_few(Xq, Xs, Wq, Ws, Y, M, N, K, stream);
    int cus = 0;
    if (device_cu_count(&cus) != LYNX_OK) return LYNX_ERR_DEVICE;
    bool taken = false;
    const lynx_status st = launch_gemm_fp8_mid(Xq, Xs, Wq, Ws, Y, M, N, K, cus, &taken, stream);
    if (taken) return st;
    // Rounds of tiles over the compute units, each at its tile's time relative to a
    // 256 x 256 one (measured at K = 3072: 33 us; 256 x 192 0.83 of that; 128 x 128, two
    // workgroups a unit, 0.75, 0.45 with at most one).  4096 x 9216: 256 x 192 101 us,
    // 256 x 256 115; 9216 x 3072: 89 and 75; 512 x 3072: 128 x 128 14 us, 256 x 192 24.
    auto tiles = [&](int tm, int tn) { return long((M + tm - 1) / tm) * ((N + tn - 1) / tn); };
    auto rounds = [](long t, long n) { return (t + n - 1) / n; };
    const long wide = rounds(tiles(256, 256), cus) * 100, mid = rounds(tiles(256, 192), cus) * 83;
    const long t22 = tiles(128, 128);
    const long small = t22 <= cus ? 45 : rounds(t22, 2 * cus) * 75;
    if (small < wide && small < mid)
        return launch_tiled<2, 2>(Xq, Xs, Wq, Ws, Y, M, N, K, cus, stream);
    return mid < wide ? launch_tiled<4, 3>(Xq, Xs, Wq, Ws, Y, M, N, K, cus, stream)
                      : launch_tiled<4, 4>(Xq, Xs, Wq, Ws, Y, M, N, K, cus, stream);
}

}  // namespace lynx
