// Attention over tiles of 256 query rows (lynx_attention): eight waves of 32 rows, two to a
// SIMD, in two groups that alternate.  While one group multiplies - S^T = K Q^T of a tile of keys,
// and O^T += V^T P^T of the tile before - the other turns scores into weights, so that the
// matrix unit and the vector unit of a SIMD both have work all the time.  A barrier ends
// each of these slots; group 1 runs one slot behind group 0: it multiplies tile t in slot 2 t + 1
// and weighs it in slot 2 t + 2.
//
// K and V tiles come by LDS-DMA into rings of four.  A group issues its half of K(t + 3) and
// V(t + 2) while it weighs tile t: their slots were read last, as K(t - 1) and V(t - 2), by group 1
// in slot 2 t - 1, and group 0 weighs tile t in slot 2 t + 1.  The loads are spread over the
// weighing, since they are taken in slower than a wave can issue them.  At the end of every
// slot 2 t all waves wait for all but the loads of their last weighing: K(t + 1) and V(t) are there
// when the barrier opens, a slot before group 0 multiplies them, so that each group reads its
// first operands ahead, at the end of its weighing.
//
// The weighing bounds a slot, and the board's power the clock: 16384 x 16384 x 8 heads x 128 942 us, 1167
// TFLOP/s, the matrix cores busy 61% of the cycles at 1.84 GHz of 2.4 (tiles of 128 rows: 1058 us).  Measured and not kept: 64 rows to a
// wave, which halves the reads from LDS, but does not fit 256 registers (accumulators in the other
// half are copied for every factor); priorities of waves (no difference); loads inside the
// multiplying (4608 x 4608 x 24 heads 290 us instead of 257).  The causal form sets registers aside
// in memory once, before the tiles with hidden keys.
#include "lynx_attn_wave.h"
#include "lynx_tile.h"

namespace lynx {
namespace {

constexpr int BMR = 256, RING = 4;

// Ends a slot: neither kind of work moves into the next one.
__device__ __forceinline__ void slot_barrier() {
    __builtin_amdgcn_sched_barrier(0);
    block_barrier();
    __builtin_amdgcn_sched_barrier(0);
}

template <int DP, bool LSE, bool CAUSAL>
__global__ __launch_bounds__(512, 2) void attn_wide_kernel(const AttnArgs A) {
    constexpr int BN = kKeys<DP>, TILE = BN * kRow<DP>;
    __shared__ __attribute__((aligned(1024))) char smem[2 * RING * TILE];
    const uint32_t lds0 = lds_addr(smem);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int group = wave >> 2;

    AttnItem w;
    if (!attn_item<BMR, BN>(A, int(blockIdx.x), w)) return;
    const AttnSpan<BMR, BN> span(A, w);
    const int row0 = w.tile * BMR + wave * 32, n = span.n;
    TileStream<DP, BN, 8, RING, false> ks;
    TileStream<DP, BN, 8, RING, true> vs;
    open_stream(ks, A, w, span, false, 0, lds0, wave, lane);
    open_stream(vs, A, w, span, true, 0, lds0 + RING * TILE, wave, lane);
    ks.issue(A.D, wave, lane);
    vs.issue(A.D, wave, lane);
    ks.issue(A.D, wave, lane);
    vs.issue(A.D, wave, lane);
    ks.issue(A.D, wave, lane);

    AttnTile<DP, BN, LSE> W;
    {
        int token, head;
        const bool valid = attn_row(A, w, row0 + (lane & 31), token, head);
        W.init(valid ? A.q + attn_q_offset(A, token, head) : nullptr, A.D);
    }
    const AttnView view(A, w, row0, lane);
    const int nw = view.tiles(span), np = CAUSAL ? min(nw, view.plain(span)) : nw;
    const uint32_t ka = W.k_first(), va = W.v_first() + RING * TILE;
    constexpr int PER = ks.PER, EACH = 2 * PER;  // loads of K and V of a tile
    auto load = [&](auto& st, int part) {        // one of two halves
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < PER; ++i)
            if (i * 2 / PER == part) st.piece(i);
        __builtin_amdgcn_sched_barrier(0);
    };
    auto weigh = [&](int t) {
        ks.begin(A.D, wave, lane);
        vs.begin(A.D, wave, lane);
        const int j = span.j0 + t, key0 = span.key(j);
        const bool pre = j < span.tp;
        if (key0 + BN > (pre ? A.prefix : view.all)) W.hide(key0, pre ? A.prefix : view.seen);
        load(ks, 0);
        const float top = W.maximum(W.s, A.c);
        load(ks, 1);
        W.relate(top, A.c);
        typename decltype(W)::Sums sum;
#pragma unroll
        for (int b = 0; b < W.NB; ++b) {
            W.weights(W.s[b], A.c, W.p[b], sum);
            if (b % (W.NB / 2) == 0) load(vs, b / (W.NB / 2));
        }
        W.add(sum);
        // here, not after the barrier: its only use is far away
        asm volatile("" : "+v"(W.l));
    };
    auto m_end = [&] {
        if (group == 0) wait_vmcnt<EACH>();
        slot_barrier();
    };
    auto w_end = [&] {
        if (group == 1) wait_vmcnt<EACH>();
        slot_barrier();
    };

    // everything, q too: where the compiler knows of loads of q under way it waits for all loads
    // before every product
    wait_vmcnt<0>();
    slot_barrier();
    if (group == 1) slot_barrier();
    int t = 0;
    uint32_t at = 0;  // of K(t) and V(t) in their rings
    if (nw > 0) {
        W.template ahead<true, false>(smem, ka, va);
        W.template multiply<true, false>(smem, ka, va);
    }
    m_end();
    if (nw > 0) {
        while (t + 1 < nw && t < np) {
            weigh(t);
            const uint32_t next = (at + TILE) & (RING * TILE - 1);
            W.template ahead<true, true>(smem, ka + next, va + at);
            w_end();
            W.template multiply<true, true>(smem, ka + next, va + at);
            m_end();
            at = next;
            ++t;
        }
        // tiles that not all rows see whole, and the last one's values
        for (; t < nw; ++t) {
            weigh(t);
            const uint32_t next = (at + TILE) & (RING * TILE - 1);
            w_end();
            if (CAUSAL && t >= np) {
                W.multiply_hidden(smem, va + at, view.seen - span.key(span.j0 + t));
            } else {
                W.template ahead<false, true>(smem, ka, va + at);
                W.template multiply<false, true>(smem, ka, va + at);
            }
            if (t + 1 < nw) {
                W.template ahead<true, false>(smem, ka + next, va);
                W.template multiply<true, false>(smem, ka + next, va);
            }
            m_end();
            at = next;
        }
    }
    for (; t < n; ++t) {  // tiles that only other waves work on
        ks.issue(A.D, wave, lane);
        vs.issue(A.D, wave, lane);
        w_end();
        m_end();
    }
    if (group == 0) slot_barrier();
    wait_vmcnt<0>();  // loads into LDS end before the workgroup does

    store_rows<DP, LSE>(A, w, W, row0, A.slots > 0 && (A.force_part || w.chunks > 1));
}

}  // namespace

lynx_status launch_attn_wide(const AttnArgs& a, int grid, hipStream_t stream) {
    const dim3 g{unsigned(grid)}, block{512};
    auto go = [&](auto dp, auto lse, auto causal) {
        hipLaunchKernelGGL((attn_wide_kernel<dp, lse, causal>), g, block, 0, stream, a);
    };
    attn_variant(a, go);
    return launch_status();
}

}  // namespace lynx
