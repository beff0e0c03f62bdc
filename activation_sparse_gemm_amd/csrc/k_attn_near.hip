// Attention on few keys (lynx_attention): all of a sequence's keys and values of a head lie in LDS,
// at most five tiles, and eight waves, two to a SIMD, walk query rows, 32 at a time, each at its own
// pace.  After the keys have come no wave waits for another, or for loads: a wave reads its next
// rows of Q while it works on the present ones, and multiplies the first tile's scores of the next
// rows together with the last tile's values of the present ones.
//
// 2 x 4096 rows on 300 keys, 16 x 72: 25 us, of which 5 until the keys are there and 14 for two row tiles to a
// wave (tiles of 128 rows, that each fetch the keys: 34); 20000 on 300, 28/4 x 128: 117 us, 737 TFLOP/s
// (179).  Two waves of a SIMD take 3500 cycles for a step each (96 channels), the products of it 1584 and
// the weights 1800: nothing makes the waves alternate, and priorities made no difference.
#include "lynx_attn_wave.h"
#include "lynx_tile.h"

namespace lynx {
namespace {

constexpr int BMR = 256;  // rows at a time

// Workgroup share * pairs + pair works on the share's row tiles of a sequence and key head.
template <int DP, bool LSE>
__global__ __launch_bounds__(512, 2) void attn_near_kernel(const AttnArgs A) {
    constexpr int BN = kKeys<DP>, TILE = BN * kRow<DP>, RING = kNearTiles;
    __shared__ __attribute__((aligned(1024))) char smem[2 * RING * TILE];
    const uint32_t lds0 = lds_addr(smem);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));

    const int pairs = A.batch * A.kv_heads;
    const int share = sgpr(int(blockIdx.x) / pairs), pair = int(blockIdx.x) - share * pairs;
    AttnItem w = {};
    w.seq = sgpr(pair / A.kv_heads);
    w.kvh = pair - w.seq * A.kv_heads;
    w.q0 = w.seq * A.len_q;
    w.lq = A.len_q;
    w.lk = A.len_k;
    w.chunks = 1;
    const AttnSpan<BMR, BN> span(A, w);
    TileStream<DP, BN, 8, RING, false> ks;
    TileStream<DP, BN, 8, RING, true> vs;
    open_stream(ks, A, w, span, false, 0, lds0, wave, lane);
    open_stream(vs, A, w, span, true, 0, lds0 + RING * TILE, wave, lane);
    for (int t = 0; t < span.n; ++t) {
        ks.issue(A.D, wave, lane);
        vs.issue(A.D, wave, lane);
    }

    const int tiles = (w.lq * A.group + 31) >> 5;
    const int per = sgpr((tiles + A.pieces - 1) / A.pieces), end = min(tiles, (share + 1) * per);
    int tile = share * per + wave;
    AttnTile<DP, BN, LSE> W;
    auto row = [&](int of) -> const uint16_t* {
        int token, head;
        const bool valid = attn_row(A, w, of * 32 + (lane & 31), token, head);
        return valid && of < end ? A.q + attn_q_offset(A, token, head) : nullptr;
    };
    W.init(row(tile), A.D);
    const uint32_t ka = W.k_first(), va = W.v_first() + RING * TILE;
    auto weigh = [&](int t) {
        if ((t + 1) * BN > w.lk) W.hide(t * BN, w.lk);
        W.relate(W.maximum(W.s, A.c), A.c);
        typename decltype(W)::Sums sum;
#pragma unroll
        for (int b = 0; b < W.NB; ++b) W.weights(W.s[b], A.c, W.p[b], sum);
        W.add(sum);
    };
    wait_vmcnt<0>();
    block_barrier();
    if (tile >= end) return;

    W.template ahead<true, false>(smem, ka, va);
    W.template multiply<true, false>(smem, ka, va);
    uint32_t at;  // of the tile in its ring
    for (;;) {
        bf16x8 next[W.KS];
        W.read_q(next, row(tile + 8), A.D);
        weigh(0);
        at = 0;
        for (int t = 1; t < span.n; ++t) {
            W.template ahead<true, true>(smem, ka + at + TILE, va + at);
            W.template multiply<true, true>(smem, ka + at + TILE, va + at);
            weigh(t);
            at += TILE;
        }
        if (tile + 8 >= end) break;
#pragma unroll
        for (int i = 0; i < W.KS; ++i) W.q[i] = next[i];
        W.template ahead<true, true>(smem, ka, va + at);
        W.template multiply<true, true>(smem, ka, va + at);
        store_rows<DP, LSE>(A, w, W, tile * 32, false);
        W.clear();
        tile += 8;
    }
    W.template ahead<false, true>(smem, ka, va + at);
    W.template multiply<false, true>(smem, ka, va + at);
    store_rows<DP, LSE>(A, w, W, tile * 32, false);
}

}  // namespace

lynx_status launch_attn_near(const AttnArgs& a, int grid, hipStream_t stream) {
    const dim3 g{unsigned(grid)}, block{512};
    auto go = [&](auto dp, auto lse) {
        hipLaunchKernelGGL((attn_near_kernel<dp, lse>), g, block, 0, stream, a);
    };
    attn_variant(a, [&](auto dp, auto lse, auto) { go(dp, lse); });
    return launch_status();
}

}  // namespace lynx
