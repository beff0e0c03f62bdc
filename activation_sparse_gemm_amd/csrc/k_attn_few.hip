// Attention of few query rows to a key head (lynx_attention): single tokens on caches.  The
// keys' and values' bytes bound it.  A workgroup holds 32 query rows (tokens x heads in
// group), its four waves take 32 keys each of a tile of 128 and add up their results at the
// end.  Each wave stages its own keys, two tiles ahead of each other, and waits for no other
// wave before the end.
#include "lynx_attn_wave.h"
#include "lynx_tile.h"

namespace lynx {
namespace {

constexpr int BN = 128, BMR = 32;

template <int DP, bool LSE>
__global__ __launch_bounds__(256, 1) void attn_few_kernel(const AttnArgs A) {
    constexpr int TILE = 32 * DP * 2;  // a wave's K (or V) of a tile
    constexpr int REGS = DP / 2;       // accumulators of a lane
    __shared__ __attribute__((aligned(1024))) char smem[4 * 4 * TILE];
    __shared__ float stat[3][4][32];
    const int lane = threadIdx.x & 63;
    const int wave = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const uint32_t mine = uint32_t(wave) * (4 * TILE);
    const uint32_t lds0 = lds_addr(smem) + mine;

    AttnWork<BMR, BN> work(A);
    AttnItem w;
    while (work.next(w)) {
        AttnPlan<BMR, BN> plan(A, w.lq, w.lk);
        plan.per = sgpr(plan.per);
        const int tp = (A.prefix + BN - 1) / BN;
        const int last_token = min(w.lq - 1, sgpr((w.tile * BMR + BMR - 1) / A.group));
        const int own = A.causal ? clampi(last_token + w.lk - w.lq + 1, 0, w.lk) : w.lk;
        const int tend = tp + (own + BN - 1) / BN;
        const int j0 = w.chunk * plan.per, j1 = min(j0 + plan.per, tend);

        AttnWave<DP, 1, LSE> W;
        W.init(lane);
        int token, head;
        const bool valid = attn_row(A, w, w.tile * BMR + (lane & 31), token, head);
        W.load_q(0, valid ? A.q + attn_q_offset(A, token, head) : nullptr, A.D);
        const int seen = A.causal ? clampi(token - w.q0 + w.lk - w.lq + 1, 0, w.lk) : w.lk;
        const int first_token = sgpr(w.tile * BMR / A.group);
        const int all = A.causal ? clampi(first_token + w.lk - w.lq + 1, 0, w.lk) : w.lk;

        const uint16_t* kb = A.k + (A.cu_k ? w.k0 * A.k_t : w.seq * A.k_b) + w.kvh * A.k_h;
        const uint16_t* vb = A.v + (A.cu_k ? w.k0 * A.v_t : w.seq * A.v_b) + w.kvh * A.v_h;
        const uint16_t* pkb = A.pk + w.kvh * A.pk_h;
        const uint16_t* pvb = A.pv + w.kvh * A.pv_h;
        AttnStage<DP, 32, 1, false> sk;
        AttnStage<DP, 32, 1, true> sv;
        bool in_prefix = false;
        auto issue = [&](int j) {
            const bool pre = j < tp;
            if (j == j0 || pre != in_prefix) {
                sk.init(pre ? A.pk_t : A.k_t, A.D, 0, lane);
                sv.init(pre ? A.pv_t : A.v_t, A.D, 0, lane);
                in_prefix = pre;
            }
            const int64_t first = int64_t(pre ? j : j - tp) * BN + 32 * wave;
            const int rows = int((pre ? A.prefix : w.lk) - first);
            const uint32_t lds = lds0 + uint32_t(j & 1) * (2 * TILE);
            sk.load((pre ? pkb : kb) + first * (pre ? A.pk_t : A.k_t), rows, A.D, lds, 0);
            sv.load((pre ? pvb : vb) + first * (pre ? A.pv_t : A.v_t), rows, A.D, lds + TILE, 0);
        };

        constexpr int LOADS = 2 * (TILE / 1024);
        if (j0 < j1) issue(j0);
        for (int j = j0; j < j1; ++j) {
            if (j + 1 < j1) {
                issue(j + 1);
                wait_vmcnt<LOADS>();
            } else {
                wait_vmcnt<0>();
            }
            asm volatile("" ::: "memory");
            const bool pre = j < tp;
            const int key0 = (pre ? j : j - tp) * BN + 32 * wave;
            const uint32_t at = mine + uint32_t(j & 1) * (2 * TILE);
            f32x16 s[1][1];
            W.scores(smem, at, 0, s[0]);
            if (key0 + 32 > (pre ? A.prefix : all)) W.mask(s[0][0], key0, pre ? A.prefix : seen);
            W.template softmax<1>(0, s, A.c);
            W.accumulate(smem, at + TILE, 0, s[0]);
            wait_lgkm0();  // the slot's reads are done before it is filled again
            asm volatile("" ::: "memory");
        }

        // the waves' results: m and l, then o by registers, which lie in a wave's own part
        const float l = W.both_sum(W.l[0]), le = LSE ? W.both_sum(W.exact[0]) : 0.f;
        if (W.h == 0) {
            stat[0][wave][lane] = W.m[0];
            stat[1][wave][lane] = l;
            if constexpr (LSE) stat[2][wave][lane] = le;
        }
        float* mo = reinterpret_cast<float*>(smem + mine);
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) mo[(16 * d + e) * 64 + lane] = W.o[0][d][e];
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
                const float* p = reinterpret_cast<const float*>(smem + i * (4 * TILE)) + 4 * g * 64 + lane;
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
            if (A.slots > 0 && w.chunk == 0) A.part_n[row] = w.chunks;
        }
        __syncthreads();  // before the next piece's keys overwrite the results
    }
}

}  // namespace

lynx_status launch_attn_few(const AttnArgs& a, int grid, hipStream_t stream) {
    const dim3 g{unsigned(grid)}, block{256};
    if (a.lse) {
        if (a.D <= 64) hipLaunchKernelGGL((attn_few_kernel<64, true>), g, block, 0, stream, a);
        else hipLaunchKernelGGL((attn_few_kernel<128, true>), g, block, 0, stream, a);
    } else {
        if (a.D <= 64) hipLaunchKernelGGL((attn_few_kernel<64, false>), g, block, 0, stream, a);
        else hipLaunchKernelGGL((attn_few_kernel<128, false>), g, block, 0, stream, a);
    }
    return launch_status();
}

}  // namespace lynx
