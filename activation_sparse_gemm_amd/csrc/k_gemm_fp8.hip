// Tiled 8-bit GEMM: Y = sum over K blocks of 2^(ex + ew) (Xq Wq^T), e4m3
// operands with E8M0 block scales, bf16 out (lynx.h).  The instruction and its
// rounding are described in k_gemm_fp8_split.hip.
//
// Persistent workgroups of 4 waves walk tiles of 64 NA x 64 NB, each wave
// 32 NA x 32 NB of it as NA x NB accumulators of 32 x 32.  A stage is 64
// channels: 64-byte rows of X and W (swizzled) and the rows' scale words, moved
// to LDS by DMA into a ring of 4 slots.  The ring is one stream of stages over
// all of a workgroup's tiles: the loads run 4 stages ahead, so those of a tile's
// last 4 stages are the next tile's first, in flight during the epilogue.  A tile
// has an even number of stages, at least 4: K % 128 == 64 and K < 256 are filled
// up with stages that load the last channels again, under scales of 2^-127 for
// both operands, whose products are zero in fp32.
//
// A stage's fragments are read from LDS into registers during the stage before
// it (two sets, 32 bytes of a row per lane and 32 x 32 block), so a stage has
// one barrier: after it, stage u + 1 has landed for all waves and slot u % 4,
// whose fragments are in registers, may be filled with stage u + 4.  With
// NA = NB = 4 a stage is 16 instructions of 64 cycles a wave, 64 KB of LDS reads
// (512 cycles at 128 B) and 33 KB of LDS writes: LDS traffic, not the matrix
// cores, limits how evenly the instructions can be fed.
//
// Scales: lane l's A operand is row l % 32, its scale the byte of the stage's K
// block in that row's word (4 blocks); a 32-column block of W lies in one
// 128-row scale block, so its scale is uniform and comes through the scalar
// cache.
#include <type_traits>

#include "lynx_fp8.h"
#include "lynx_tile.h"

namespace lynx {
namespace {

// Edge tiles: each lane stores its own column, where it lies inside N; rows past
// M lie past the end of the buffer (see store_block_direct).
template <int NB, int NA>
__device__ __forceinline__ void store_block_edge(const f32x16 (&acc)[NA][NB],
                                                 __amdgpu_buffer_rsrc_t rsY, int N, int row0,
                                                 int col0) {
    const int l = fresh_lane();
    const int r = l & 31, h = l >> 5;
#pragma unroll
    for (int b = 0; b < NB; ++b) {
        const int col = col0 + 32 * b + r;
        if (col < N) {
#pragma unroll
            for (int a = 0; a < NA; ++a)
#pragma unroll
                for (int e = 0; e < 16; ++e) {
                    const int row = row0 + 32 * a + 8 * (e / 4) + 4 * h + e % 4;
                    __builtin_amdgcn_raw_buffer_store_b16(
                        __builtin_bit_cast(uint16_t, static_cast<__bf16>(acc[a][b][e])), rsY,
                        (uint32_t(row) * uint32_t(N) + uint32_t(col)) * 2u, 0, 0);
                }
        }
    }
}

template <int NA, int NB>
__global__ __launch_bounds__(NT, NA == 4 ? 1 : 2) void gemm_fp8_tiled(
    const uint8_t* __restrict__ Xq, const uint8_t* __restrict__ Xs,
    const uint8_t* __restrict__ Wq, const uint32_t* __restrict__ Ws, uint16_t* __restrict__ Y,
    int M, int N, int K) {
    constexpr int TM = 64 * NA, TN = 64 * NB;
    constexpr int kRow = 64;                        // LDS bytes per row and stage
    constexpr int kA = TM * kRow, kB = TN * kRow;
    constexpr int kStage = kA + kB + 1024;          // + a scale word per row (256 places)
    constexpr int kSlots = 4;
    constexpr int kDma = NA + NB + 1;               // DMA instructions per wave and stage
    constexpr int kM = NA * NB;                     // matrix instructions per wave and stage
    constexpr int kReads = 2 * (NA + NB);           // 16-byte LDS reads per wave and stage
    constexpr int kBar = 1;                         // the barrier follows instruction kBar
    constexpr uint32_t kPast = 0xFFFFFF00u;         // past the end of every buffer (< 2^31 bytes)
    constexpr int kBS = NB == 3 ? NB : 1;           // scale blocks a wave's columns touch
    static_assert(kSlots * kStage <= 160 * 1024 / (NA == 4 ? 1 : 2), "LDS budget");
    __shared__ __attribute__((aligned(1024))) char smem[kSlots * kStage];

    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int r = lane & 31, h = lane >> 5;
    const int wm = wave & 1, wn = wave >> 1;
    const int tiles_m = (M + TM - 1) / TM, tiles_n = (N + TN - 1) / TN;
    const int ntiles = tiles_m * tiles_n;
    const int real = K / 64;                       // stages that hold channels of K
    const int nk = max((real + 1) & ~1, kSlots);
    const int words = fp8_scale_words(K);
    const int nblocks = (N + kFp8Block - 1) / kFp8Block;

    // ---- producer: DMA instruction j of wave w moves rows 16 (w + 4j) + l/4 of an
    // operand, lane l's 16 bytes the chunk that the row's swizzle puts there
    const uint32_t lds0 = lds_addr(smem);
    const i32x4 rsA = make_rsrc(Xq, uint32_t(M) * uint32_t(K));
    const i32x4 rsB = make_rsrc(Wq, uint32_t(N) * uint32_t(K));
    const i32x4 rsS = make_rsrc(Xs, uint32_t(words) * uint32_t(M) * 4u);
    uint32_t voffA[NA], voffB[NB], voffS;
    auto aim = [&](int v) {  // at tile v, or past the last tile
        if (v >= ntiles) {
            // the loads go on, so that every wait has the same count, but from past
            // the ends of the buffers: they read nothing
#pragma unroll
            for (int j = 0; j < NA; ++j) voffA[j] = kPast;
#pragma unroll
            for (int j = 0; j < NB; ++j) voffB[j] = kPast;
            voffS = kPast;
            return;
        }
        int tm, tn;
        tile_of(v, tiles_m, tiles_n, tm, tn);
        const int l = fresh_lane();
#pragma unroll
        for (int j = 0; j < NA; ++j) {
            const int row = 16 * (wave + 4 * j) + (l >> 2);
            voffA[j] = uint32_t(tm * TM + row) * uint32_t(K) + uint32_t(16 * ((l & 3) ^ swz64(row)));
        }
#pragma unroll
        for (int j = 0; j < NB; ++j) {
            const int row = 16 * (wave + 4 * j) + (l >> 2);
            voffB[j] = uint32_t(tn * TN + row) * uint32_t(K) + uint32_t(16 * ((l & 3) ^ swz64(row)));
        }
        // the word offset goes into the scalar part, which is not range checked:
        // rows past the end take the last row's words
        voffS = uint32_t(min(tm * TM + 64 * (wave % NA) + l, M - 1)) * 4u;
    };
    // DMA instruction i of stage t of the tile aimed at
    auto dma = [&](int slot, int t, int i) {
        const uint32_t base = lds0 + uint32_t(slot);
        const uint32_t ko = uint32_t(min(t, real - 1)) * kRow;
        if (i < NA)
            dma16(base + 1024 * (wave + 4 * i), voffA[i], rsA, ko);
        else if (i < NA + NB)
            dma16(base + kA + 1024 * (wave + 4 * (i - NA)), voffB[i - NA], rsB, ko);
        else
            dma4(base + kA + kB + 256 * wave, voffS, rsS, (ko >> 9) * uint32_t(M) * 4u);
    };

    // ---- consumer
    const int s64 = swz64(r);
    const int offA = (wm * 32 * NA + r) * kRow, offB = kA + (wn * 32 * NB + r) * kRow;
    const int offS = kA + kB + (wm * 32 * NA + r) * 4;
    struct Frags {
        i32x4 a[NA][2], b[NB][2];
    };
    Frags fr[2];
    uint32_t sa[NA], sb[kBS];  // scale words of the stage (and of what follows in its tile)
    auto read_n = [&](int slot, Frags& f, int n) {
        const int blk = n >> 1, part = n & 1;
        const int c = 16 * ((2 * part + h) ^ s64);
        if (blk < NA)
            f.a[blk][part] = lds_read<i32x4>(smem + slot, offA + blk * 32 * kRow + c);
        else
            f.b[blk - NA][part] = lds_read<i32x4>(smem + slot, offB + (blk - NA) * 32 * kRow + c);
    };
    auto read_scales = [&](int slot, uint32_t* s) {
#pragma unroll
        for (int a = 0; a < NA; ++a) s[a] = lds_read<uint32_t>(smem + slot, offS + a * 128);
    };
    f32x16 acc[NA][NB];
    auto mma = [&](const Frags& f, int k, int shift, uint32_t keep) {
        const int a = k % NA, b = k / NA;
        const i32x8 va = __builtin_shufflevector(f.a[a][0], f.a[a][1], 0, 1, 2, 3, 4, 5, 6, 7);
        const i32x8 vb = __builtin_shufflevector(f.b[b][0], f.b[b][1], 0, 1, 2, 3, 4, 5, 6, 7);
        acc[a][b] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
            va, vb, acc[a][b], 0, 0, 0, int((sa[a] >> shift) & keep), 0,
            int((sb[kBS == 1 ? 0 : b] >> shift) & keep));
    };
    int cur = 0;  // slot of the stage at hand
    auto next_slot = [](int s) { return s + kStage == kSlots * kStage ? 0 : s + kStage; };
    // stage t: its instructions, the next stage's LDS reads (its scale words too
    // where it opens a block), and the loads of stage `lt` into the slot it frees
    auto stage = [&](auto set, auto opens, int t, int lt, uint32_t* sn) {
        constexpr int S = decltype(set)::value;
        const int nxt = next_slot(cur);
        const int shift = 8 * ((t >> 1) & 3);             // its block's byte in the scale words
        const uint32_t keep = t < real ? 0xFFu : 0u;      // 2^-127 for a filled-up stage
        constexpr int kAfter = kM - kBar - 1;  // instructions after the barrier
#pragma unroll
        for (int k = 0; k < kM; ++k) {
            mma(fr[S], k, shift, keep);
            if (k == kBar) {
                wait_vmcnt_lgkm0<2 * kDma>();
                block_barrier();
                if constexpr (decltype(opens)::value) read_scales(nxt, sn);
            }
            if (k > kBar) {
                const int q = k - kBar - 1;
#pragma unroll
                for (int n = q * kReads / kAfter; n < (q + 1) * kReads / kAfter; ++n)
                    read_n(nxt, fr[1 - S], n);
#pragma unroll
                for (int i = q * kDma / kAfter; i < (q + 1) * kDma / kAfter; ++i) dma(cur, lt, i);
            }
            __builtin_amdgcn_sched_barrier(0);
        }
        cur = nxt;
    };

    aim(blockIdx.x);
    for (int u = 0; u < kSlots; ++u)
#pragma unroll
        for (int i = 0; i < kDma; ++i) dma(u * kStage, u, i);
    wait_vmcnt<3 * kDma>();
    block_barrier();
    read_scales(0, sa);
#pragma unroll
    for (int n = 0; n < kReads; ++n) read_n(0, fr[0], n);

    const __amdgpu_buffer_rsrc_t rsY =
        __builtin_amdgcn_make_buffer_rsrc(Y, 0, int(uint32_t(M) * uint32_t(N) * 2u), kRsrcWord3);
    for (int v = blockIdx.x; v < ntiles; v += gridDim.x) {
        int tm, tn;
        tile_of(v, tiles_m, tiles_n, tm, tn);
        const int row0 = tm * TM + wm * 32 * NA, col0 = tn * TN + wn * 32 * NB;
        const uint32_t* wsp[kBS];
#pragma unroll
        for (int b = 0; b < kBS; ++b)
            wsp[b] = Ws + size_t(__builtin_amdgcn_readfirstlane(
                              min((col0 + 32 * b) / kFp8Block, nblocks - 1))) * size_t(words);
#pragma unroll
        for (int b = 0; b < kBS; ++b) sb[b] = wsp[b][0];
#pragma unroll
        for (int a = 0; a < NA; ++a)
#pragma unroll
            for (int b = 0; b < NB; ++b) acc[a][b] = f32x16{};

        uint32_t sn[NA], bn[kBS];
        using Set0 = std::integral_constant<int, 0>;
        using Set1 = std::integral_constant<int, 1>;
        auto fetch = [&](int t) {  // W's scale words of stage t, t + 1 opening a block
            const int w = min(t >> 3, words - 1);
#pragma unroll
            for (int b = 0; b < kBS; ++b) bn[b] = wsp[b][w];
        };
        auto take = [&] {
#pragma unroll
            for (int a = 0; a < NA; ++a) sa[a] = sn[a];
#pragma unroll
            for (int b = 0; b < kBS; ++b) sb[b] = bn[b];
        };
        auto pair = [&](int t, int lt) {  // a block of 128 channels, loading lt and lt + 1
            fetch(t + 2);
            stage(Set0{}, std::false_type{}, t, lt, sn);
            stage(Set1{}, std::true_type{}, t + 1, lt + 1, sn);
            take();
        };
        int t = 0;
        for (; t < nk - 4; t += 2) pair(t, t + 4);
        aim(v + int(gridDim.x));
        for (; t < nk; t += 2) pair(t, t + 4 - nk);
        if ((N & 1) == 0 && tn * TN + TN <= N) store_block_direct<NB>(acc, rsY, N, row0, col0);
        else store_block_edge<NB>(acc, rsY, N, row0, col0);
    }
    wait_vmcnt<0>();  // the loads past the last tile still write LDS
}

template <int NA, int NB>
lynx_status launch_tiled(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                         const uint8_t* Ws, uint16_t* Y, int M, int N, int K, int cus,
                         hipStream_t stream) {
    const long tiles = long((M + 64 * NA - 1) / (64 * NA)) * ((N + 64 * NB - 1) / (64 * NB));
    const long most = long(cus) * (NA == 4 ? 1 : 2);
    hipLaunchKernelGGL((gemm_fp8_tiled<NA, NB>), dim3(unsigned(tiles < most ? tiles : most)),
                       dim3(NT), 0, stream, Xq, Xs, Wq, reinterpret_cast<const uint32_t*>(Ws), Y,
                       M, N, K);
    return launch_status();
}

}  // namespace

lynx_status launch_gemm_fp8(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                            const uint8_t* Ws, uint16_t* Y, int M, int N, int K,
                            hipStream_t stream) {
    if (M <= 64) return launch_gemm_fp8_split(Xq, Xs, Wq, Ws, Y, M, N, K, stream);
    int cus = 0;
    if (device_cu_count(&cus) != LYNX_OK) return LYNX_ERR_DEVICE;
    auto tiles = [&](int tm, int tn) { return long((M + tm - 1) / tm) * ((N + tn - 1) / tn); };
    if (tiles(256, 256) >= cus / 2) {
        auto cost = [&](int tn) { return (tiles(256, tn) + cus - 1) / cus * tn; };
        return cost(192) < cost(256)
                   ? launch_tiled<4, 3>(Xq, Xs, Wq, Ws, Y, M, N, K, cus, stream)
                   : launch_tiled<4, 4>(Xq, Xs, Wq, Ws, Y, M, N, K, cus, stream);
    }
    if (tiles(128, 128) >= cus / 2)
        return launch_tiled<2, 2>(Xq, Xs, Wq, Ws, Y, M, N, K, cus, stream);
    return launch_gemm_fp8_split(Xq, Xs, Wq, Ws, Y, M, N, K, stream);
}

}  // namespace lynx
