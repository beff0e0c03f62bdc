// Attention over tiles of 128 query rows (lynx_attention): four waves of 32 rows walk the keys
// together, and two such workgroups share a compute unit, so that one's products and another's
// weights keep the matrix and the vector unit of a SIMD busy together.
//
// A step multiplies S^T = K Q^T of tile t with O^T += V^T P^T of tile t - 1, then turns tile t's
// scores into weights.  K and V tiles come by LDS-DMA into rings of two: on top of step t all waves
// meet, K(t - 1) and V(t - 2) have been read, and K(t + 1) and V(t) are issued into their slots.
//
// The matrix unit's and the vector unit's time together bound it: two waves of a SIMD take 3700
// cycles for a step each (128 channels), of which products fill 2112, since nothing makes the two alternate.
// 4 x 1024 queries on a prefix of 2560 and their own keys, 24 x 128: 186 us, 970 TFLOP/s, the matrix
// cores busy 44% of the cycles at 2.1 GHz; 8661 tokens in 7 causal sequences, 32/8 x 128: 233 us, 860.
#pragma once

#include "lynx_attn_wave.h"
#include "lynx_tile.h"

namespace lynx {

constexpr int kTileRows = 128;

// smem: 64 KB, 1 KB aligned
template <int DP, bool LSE, bool CAUSAL>
__device__ __forceinline__ void attn_tile(const AttnArgs& A, int block, char* smem) {
    constexpr int BMR = kTileRows, BN = kKeys<DP>, TILE = BN * kRow<DP>;
    const uint32_t lds0 = lds_addr(smem);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));

    AttnItem w;
    if (!attn_item<BMR, BN>(A, block, w)) return;
    const AttnSpan<BMR, BN> span(A, w);
    const int row0 = w.tile * BMR + wave * 32;
    TileStream<DP, BN, 4, 2, false> ks;
    TileStream<DP, BN, 4, 2, true> vs;
    open_stream(ks, A, w, span, false, 0, lds0, wave, lane);
    open_stream(vs, A, w, span, true, 0, lds0 + 2 * TILE, wave, lane);
    ks.issue(A.D, wave, lane);

    AttnTile<DP, BN, LSE> W;
    {
        int token, head;
        const bool valid = attn_row(A, w, row0 + (lane & 31), token, head);
        W.init(valid ? A.q + attn_q_offset(A, token, head) : nullptr, A.D);
    }
    const AttnView view(A, w, row0, lane);
    const int nw = view.tiles(span), np = CAUSAL ? min(nw, view.plain(span)) : nw;
    const uint32_t ka = W.k_first(), va = W.v_first() + 2 * TILE;
    auto weigh = [&](int t) {
        const int j = span.j0 + t, key0 = span.key(j);
        const bool pre = j < span.tp;
        if (key0 + BN > (pre ? A.prefix : view.all)) W.hide(key0, pre ? A.prefix : view.seen);
        W.relate(W.maximum(W.s, A.c), A.c);
        typename decltype(W)::Sums sum;
#pragma unroll
        for (int b = 0; b < W.NB; ++b) W.weights(W.s[b], A.c, W.p[b], sum);
        W.add(sum);
    };

    // K(0), and q: where the compiler knows of loads of q under way it waits for all loads
    // before every product
    wait_vmcnt<0>();
    block_barrier();
    // The loads of a step are spread over its products: a unit takes 64 bytes a clock, so the four
    // waves' 32 loads at once hold up each wave for 500 cycles
    auto loads = [&](int i) {
        constexpr int PER = ks.PER;
        if (i == 0) ks.begin(A.D, wave, lane);
        if (i == 1) vs.begin(A.D, wave, lane);
#pragma unroll
        for (int n = 0; n < 2 * PER; ++n)
            if (i == 1 + n * (W.NM - 1) / (2 * PER)) n < PER ? ks.piece(n) : vs.piece(n - PER);
    };
    if (nw > 0) {
        W.template ahead<true, false>(smem, ka, va);
        W.template multiply<true, false>(smem, ka, va, loads);
        weigh(0);
    } else {
        ks.issue(A.D, wave, lane);
        vs.issue(A.D, wave, lane);
    }
    auto top = [&](int t) {
        wait_vmcnt<0>();
        block_barrier();
        if (t < span.n) {
            ks.issue(A.D, wave, lane);
            vs.issue(A.D, wave, lane);
        }
    };
    uint32_t at = 0;  // of V(t - 1); K(t) has the other slot
    int t = 1;
    for (; t < nw && t <= np; ++t) {
        wait_vmcnt<0>();
        block_barrier();
        W.template ahead<true, true>(smem, ka + (TILE - at), va + at);
        W.template multiply<true, true>(smem, ka + (TILE - at), va + at, loads);
        weigh(t);
        at = TILE - at;
    }
    // tiles that not all rows see whole, and the last one's values
    for (; t <= nw; ++t) {
        top(t);
        if (CAUSAL && t > np) {
            W.multiply_hidden(smem, va + at, view.seen - span.key(span.j0 + t - 1));
        } else {
            W.template ahead<false, true>(smem, ka, va + at);
            W.template multiply<false, true>(smem, ka, va + at);
        }
        if (t == nw) break;
        W.template ahead<true, false>(smem, ka + (TILE - at), va);
        W.template multiply<true, false>(smem, ka + (TILE - at), va);
        weigh(t);
        at = TILE - at;
    }
    if (nw > 0) ++t;
    for (; t <= span.n; ++t) top(t);  // tiles that only other waves work on
    wait_vmcnt<0>();                  // loads into LDS end before the workgroup does
    store_rows<DP, LSE>(A, w, W, row0, A.slots > 0 && (A.force_part || w.chunks > 1));
}

}  // namespace lynx
