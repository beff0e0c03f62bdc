// Attention over tiles of 128 query rows (lynx_attention): a workgroup holds four waves of
// 32 rows and walks the keys in tiles of 64, which all of them read from LDS.
#include "lynx_attn_wave.h"
#include "lynx_tile.h"

namespace lynx {
namespace {

constexpr int BN = 64;

template <int DP, int QB, bool LSE>
__global__ __launch_bounds__(256, QB == 1 ? 2 : 1) void attn_tile_kernel(const AttnArgs A) {
    constexpr int BMR = 128 * QB, TILE = BN * DP * 2;
    __shared__ __attribute__((aligned(1024))) char smem[4 * TILE];  // two slots of K, two of V
    const uint32_t lds0 = lds_addr(smem);
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));

    AttnWork<BMR, BN> work(A);
    AttnItem w;
    while (work.next(w)) {
        AttnPlan<BMR, BN> plan(A, w.lq, w.lk);
        plan.per = sgpr(plan.per);
        // tiles of keys: tp of the prefix, then the sequence's own, up to the last one that the
        // row tile's last query sees
        const int tp = (A.prefix + BN - 1) / BN;
        const int last_token = min(w.lq - 1, sgpr((w.tile * BMR + BMR - 1) / A.group));
        const int own = A.causal ? clampi(last_token + w.lk - w.lq + 1, 0, w.lk) : w.lk;
        const int tend = tp + (own + BN - 1) / BN;
        const int j0 = w.chunk * plan.per, j1 = min(j0 + plan.per, tend);

        AttnWave<DP, QB, LSE> W;
        W.init(lane);
        int seen[QB], token[QB], head[QB];
        bool valid[QB];
#pragma unroll
        for (int b = 0; b < QB; ++b) {
            const int row = w.tile * BMR + wave * 32 * QB + 32 * b + (lane & 31);
            valid[b] = attn_row(A, w, row, token[b], head[b]);
            W.load_q(b, valid[b] ? A.q + attn_q_offset(A, token[b], head[b]) : nullptr, A.D);
            seen[b] = A.causal ? clampi(token[b] - w.q0 + w.lk - w.lq + 1, 0, w.lk) : w.lk;
        }
        // keys that all of the wave's rows see, and that any does
        const int wt0 = sgpr((w.tile * BMR + wave * 32 * QB) / A.group);
        const int wt1 = min(w.lq - 1, sgpr((w.tile * BMR + wave * 32 * QB + 32 * QB - 1) / A.group));
        const int all = A.causal ? clampi(wt0 + w.lk - w.lq + 1, 0, w.lk) : w.lk;
        const int any = wt0 >= w.lq ? 0 : A.causal ? clampi(wt1 + w.lk - w.lq + 1, 0, w.lk) : w.lk;

        const uint16_t* kb = A.k + (A.cu_k ? w.k0 * A.k_t : w.seq * A.k_b) + w.kvh * A.k_h;
        const uint16_t* vb = A.v + (A.cu_k ? w.k0 * A.v_t : w.seq * A.v_b) + w.kvh * A.v_h;
        const uint16_t* pkb = A.pk + w.kvh * A.pk_h;
        const uint16_t* pvb = A.pv + w.kvh * A.pv_h;
        AttnStage<DP, BN, 4, false> sk;
        AttnStage<DP, BN, 4, true> sv;
        bool in_prefix = false;
        auto issue = [&](int j) {
            const bool pre = j < tp;
            if (j == j0 || pre != in_prefix) {
                sk.init(pre ? A.pk_t : A.k_t, A.D, wave, lane);
                sv.init(pre ? A.pv_t : A.v_t, A.D, wave, lane);
                in_prefix = pre;
            }
            const int64_t first = int64_t(pre ? j : j - tp) * BN;
            const int rows = int((pre ? A.prefix : w.lk) - first);
            const uint32_t lds = lds0 + uint32_t(j & 1) * (2 * TILE);
            sk.load((pre ? pkb : kb) + first * (pre ? A.pk_t : A.k_t), rows, A.D, lds, wave);
            sv.load((pre ? pvb : vb) + first * (pre ? A.pv_t : A.v_t), rows, A.D, lds + TILE, wave);
        };

        __syncthreads();  // the slots of the piece before are free
        if (j0 < j1) issue(j0);
        for (int j = j0; j < j1; ++j) {
            wait_vmcnt<0>();
            block_barrier();
            if (j + 1 < j1) issue(j + 1);
            const bool pre = j < tp;
            const int key0 = (pre ? j : j - tp) * BN;
            const int some = pre ? A.prefix : any, every = pre ? A.prefix : all;
            if (key0 >= some || (pre && any == 0 && wt0 >= w.lq)) continue;
            const uint32_t at = uint32_t(j & 1) * (2 * TILE);
            f32x16 s[2][QB];
            W.scores(smem, at, 0, s[0]);
            W.scores(smem, at, 32, s[1]);
            if (key0 + BN > every) {
#pragma unroll
                for (int b = 0; b < QB; ++b) {
                    W.mask(s[0][b], key0, pre ? A.prefix : seen[b]);
                    W.mask(s[1][b], key0 + 32, pre ? A.prefix : seen[b]);
                }
            }
#pragma unroll
            for (int b = 0; b < QB; ++b) W.template softmax<2>(b, s, A.c);
            W.accumulate(smem, at + TILE, 0, s[0]);
            W.accumulate(smem, at + TILE, 32, s[1]);
        }

        const bool part = A.slots > 0 && (A.force_part || w.chunks > 1);
#pragma unroll
        for (int b = 0; b < QB; ++b) {
            const float l = W.both_sum(W.l[b]), le = LSE ? W.both_sum(W.exact[LSE ? b : 0]) : 0.f;
            if (!valid[b]) continue;
            const int64_t row = int64_t(token[b]) * A.heads + head[b];
            if (part) {
                const int64_t slot = row * A.slots + A.slot0 + w.chunk;
                float* o = A.part_o + slot * A.D;
#pragma unroll
                for (int d = 0; d < DP / 32; ++d)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int at = 32 * d + 8 * g + 4 * W.h;
                        if (at < A.D)
                            *reinterpret_cast<f32x4*>(o + at) =
                                f32x4{W.o[b][d][4 * g], W.o[b][d][4 * g + 1], W.o[b][d][4 * g + 2],
                                      W.o[b][d][4 * g + 3]};
                    }
                if (W.h == 0) {
                    A.part_ml[slot] = float4{W.m[b], l, le, 0.f};
                    if (w.chunk == 0) A.part_n[row] = w.chunks;
                }
            } else {
                const float inv = l == 0.f ? 0.f : 1.f / l;
                uint16_t* o = A.out + attn_o_offset(A, token[b], head[b]);
#pragma unroll
                for (int d = 0; d < DP / 32; ++d)
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const int at = 32 * d + 8 * g + 4 * W.h;
                        if (at < A.D)
                            *reinterpret_cast<u32x2*>(o + at) =
                                u32x2{pack_bf16(W.o[b][d][4 * g] * inv, W.o[b][d][4 * g + 1] * inv),
                                      pack_bf16(W.o[b][d][4 * g + 2] * inv, W.o[b][d][4 * g + 3] * inv)};
                    }
                if (W.h == 0) {
                    if constexpr (LSE) A.lse[row] = le == 0.f ? -INFINITY : (W.m[b] + log2f(le)) * kLn2;
                    if (A.slots > 0 && w.chunk == 0) A.part_n[row] = 1;
                }
            }
        }
    }
}

}  // namespace

lynx_status launch_attn_tile(const AttnArgs& a, int grid, hipStream_t stream) {
    const dim3 g{unsigned(grid)}, block{256};
    if (a.lse) {
        if (a.D <= 64) hipLaunchKernelGGL((attn_tile_kernel<64, 1, true>), g, block, 0, stream, a);
        else hipLaunchKernelGGL((attn_tile_kernel<128, 1, true>), g, block, 0, stream, a);
    } else {
        if (a.D <= 64) hipLaunchKernelGGL((attn_tile_kernel<64, 1, false>), g, block, 0, stream, a);
        else hipLaunchKernelGGL((attn_tile_kernel<128, 1, false>), g, block, 0, stream, a);
    }
    return launch_status();
}

}  // namespace lynx
