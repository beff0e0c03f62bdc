// Attention of few query rows to a key head (lynx_attention): single tokens on caches.  The
// keys' and values' bytes bound it.  A workgroup holds 32 query rows (tokens x heads in
// group), its four waves take 32 keys each of a tile of 128 and add up their results at the
// end.  Each wave stages its own keys and waits for no other wave before the end: K of the next
// tile is under way while V of this one is multiplied, and the other way round.  Two such
// workgroups share a compute unit, 64 KB of keys and values under way in each.  32 tokens on
// caches of 17 .. 16400 keys, 32/8 x 128: 1.05 GB in 197 us, 5.3 TB/s, a copy's rate.
#pragma once

#include "lynx_attn_wave.h"
#include "lynx_tile.h"

namespace lynx {

constexpr int kFewRows = 32, kFewKeys = 128;

// smem: 64 KB, 1 KB aligned
template <int DP, bool LSE, bool CAUSAL>
__device__ __forceinline__ void attn_few(const AttnArgs& A, int block, char* smem, float (&stat)[3][4][32]) {
    constexpr int BMR = kFewRows, BN = kFewKeys;
    constexpr int TILE = 32 * kRow<DP>;  // a wave's K (or V) of a tile
    constexpr int RING = 256 / kRow<DP>;
    constexpr int REGS = DP / 2;       // accumulators of a lane
    static_assert(4 * 2 * RING * TILE == 65536, "");
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const uint32_t mine = uint32_t(wave) * (2 * RING * TILE);
    const uint32_t lds0 = lds_addr(smem) + mine;

    AttnItem w;
    if (!attn_item<BMR, BN>(A, block, w)) return;
    const AttnSpan<BMR, BN> span(A, w);
    const int row0 = w.tile * BMR, n = span.n;
    TileStream<DP, 32, 1, RING, false> ks;
    TileStream<DP, 32, 1, RING, true> vs;
    open_stream(ks, A, w, span, false, 32 * wave, lds0, 0, lane);
    open_stream(vs, A, w, span, true, 32 * wave, lds0 + RING * TILE, 0, lane);
    // (where the compiler knows of loads of q under way it waits for all loads before every
    // product, so q is waited for here)
    ks.issue(A.D, 0, lane);
    vs.issue(A.D, 0, lane);
    AttnTile<DP, 32, LSE> W;
    int token, head;
    const bool valid = attn_row(A, w, row0 + (lane & 31), token, head);
    W.init(valid ? A.q + attn_q_offset(A, token, head) : nullptr, A.D);
    wait_vmcnt<0>();
#pragma unroll
    for (int i = 1; i < RING; ++i) {
        ks.issue(A.D, 0, lane);
        vs.issue(A.D, 0, lane);
    }
    const AttnView view(A, w, row0, lane);
    const uint32_t ka = mine + W.k_first(), va = mine + RING * TILE + W.v_first();
    uint32_t at = 0;
    constexpr int PER = ks.PER;
    for (int t = 0; t < n; ++t) {
        // K(t): all but V(t) and the RING - 1 tiles behind it
        wait_vmcnt<(2 * RING - 1) * PER>();
        asm volatile("" ::: "memory");
        W.template ahead<true, false>(smem, ka + at, va + at);
        W.template multiply<true, false>(smem, ka + at, va + at);
        wait_lgkm0();
        asm volatile("" ::: "memory");
        ks.issue(A.D, 0, lane);
        const int j = span.j0 + t, key0 = span.key(j) + 32 * wave;
        const bool pre = j < span.tp;
        if (key0 + 32 > (pre ? A.prefix : view.all)) W.hide(key0, pre ? A.prefix : view.seen);
        W.relate(W.maximum(W.s, A.c), A.c);
        typename decltype(W)::Sums sum;
        W.weights(W.s[0], A.c, W.p[0], sum);
        W.add(sum);
        wait_vmcnt<(2 * RING - 1) * PER>();  // V(t)
        asm volatile("" ::: "memory");
        if (CAUSAL && !pre && view.all < view.lk && key0 + 32 > view.all) {
            W.multiply_hidden(smem, va + at, view.seen - key0);
        } else {
            W.template ahead<false, true>(smem, ka + at, va + at);
            W.template multiply<false, true>(smem, ka + at, va + at);
        }
        wait_lgkm0();
        asm volatile("" ::: "memory");
        vs.issue(A.D, 0, lane);
        at = at == (RING - 1) * TILE ? 0 : at + TILE;
    }
    wait_vmcnt<0>();

    // the waves' results: m and l, then o by registers, in the wave's own part
    const float l = W.both_sum(W.l), le = LSE ? W.both_sum(W.exact) : 0.f;
    if (W.h == 0) {
        stat[0][wave][lane] = W.m;
        stat[1][wave][lane] = l;
        if constexpr (LSE) stat[2][wave][lane] = le;
    }
    float* mo = reinterpret_cast<float*>(smem + mine);
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int e = 0; e < 16; ++e) mo[(16 * d + e) * 64 + lane] = W.o[d][e];
    __syncthreads();
    float M = -INFINITY, f[4], lsum = 0.f, esum = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) M = fmaxf(M, stat[0][i][lane & 31]);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float mi = stat[0][i][lane & 31];
        f[i] = mi == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(mi - M);
        lsum += f[i] * stat[1][i][lane & 31];
        if constexpr (LSE) esum += f[i] * stat[2][i][lane & 31];
    }
    const bool part = A.slots > 0 && (A.force_part || w.chunks > 1);
    const int64_t row = int64_t(token) * A.heads + head;
    const int64_t slot = row * A.slots + A.slot0 + w.chunk;
    const float inv = part ? 1.f : lsum == 0.f ? 0.f : 1.f / lsum;
    constexpr int GROUPS = REGS / 4 / 4;  // groups of four channels that a wave finishes
#pragma unroll
    for (int gi = 0; gi < GROUPS; ++gi) {
        const int g = wave * GROUPS + gi, d = 32 * (g / 4) + 8 * (g % 4) + 4 * W.h;
        f32x4 sum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float* p = reinterpret_cast<const float*>(smem + i * (2 * RING * TILE)) + 4 * g * 64 + lane;
#pragma unroll
            for (int e = 0; e < 4; ++e) sum[e] = fmaf(f[i], p[64 * e], sum[e]);
        }
        if (valid && d < A.D) {
            if (part)
                *reinterpret_cast<f32x4*>(A.part_o + slot * A.D + d) = sum;
            else
                *reinterpret_cast<u32x2*>(A.out + attn_o_offset(A, token, head) + d) =
                    u32x2{pack_bf16(sum[0] * inv, sum[1] * inv), pack_bf16(sum[2] * inv, sum[3] * inv)};
        }
    }
    if (valid && wave == 0 && W.h == 0) {
        if (part)
            A.part_ml[slot] = float4{M, lsum, esum, 0.f};
        else if (LSE)
            A.lse[row] = esum == 0.f ? -INFINITY : (M + log2f(esum)) * kLn2;
        if (A.slots > 0 && w.chunk == 0 && A.part_n) A.part_n[row] = w.chunks;
    }
}

}  // namespace lynx
