// Joins the partial results of a row's chunks of keys (lynx_attention):
//   M = max m_i,   o = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i,   lse = (M + log2 l) ln 2 (l of unrounded weights)
// One workgroup to a row: eight groups of 32 lanes take every eighth slot, 4 channels a lane.
#include "lynx_attn.h"

namespace lynx {
namespace {

__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs A, int prefix_slots) {
    __shared__ f32x4 sum[8][32];
    __shared__ float2 stat[8];
    const int row = int(blockIdx.x), token = row / A.heads, head = row - token * A.heads;
    if (A.cu_q) {  // rows of no sequence
        if (token < A.cu_q[0] || token >= A.cu_q[A.batch]) return;
    }
    const int own = clampi(A.part_n[row], 1, A.slots - prefix_slots);
    const int n = prefix_slots + own;
    if (n == 1 && !A.force_part) return;  // written already
    const int g = threadIdx.x >> 5, c = 4 * (threadIdx.x & 31);
    const int64_t first = int64_t(row) * A.slots;
    float M = -INFINITY, l = 0.f, le = 0.f;
    for (int i = 0; i < n; ++i) M = fmaxf(M, A.part_ml[first + i].x);
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    for (int i = g; i < n; i += 8) {
        const float4 ml = A.part_ml[first + i];
        if (ml.x == -INFINITY) continue;  // no key was seen: l and o are 0
        const float f = __builtin_amdgcn_exp2f(ml.x - M);
        l = fmaf(f, ml.y, l);
        le = fmaf(f, ml.z, le);
        if (c < A.D) {
            const f32x4 p = *reinterpret_cast<const f32x4*>(A.part_o + (first + i) * A.D + c);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] = fmaf(f, p[e], o[e]);
        }
    }
    sum[g][threadIdx.x & 31] = o;
    if ((threadIdx.x & 31) == 0) stat[g] = float2{l, le};
    __syncthreads();
    if (g != 0) return;
    l = le = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        l += stat[i].x;
        le += stat[i].y;
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
        o[e] = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) o[e] += sum[i][threadIdx.x][e];
        o[e] *= inv;
    }
    if (c < A.D) {
        const int b = token / A.addr_len;
        uint16_t* p = A.out + b * A.o_b + (token - b * A.addr_len) * A.o_t + head * A.o_h;
        *reinterpret_cast<u32x2*>(p + c) = u32x2{pack_bf16(o[0], o[1]), pack_bf16(o[2], o[3])};
    }
    if (A.lse && threadIdx.x == 0) A.lse[row] = le == 0.f ? -INFINITY : (M + log2f(le)) * kLn2;
}

}  // namespace

lynx_status launch_attn_join(const AttnArgs& a, int prefix_slots, hipStream_t stream) {
    hipLaunchKernelGGL(attn_join_kernel, dim3(unsigned(int64_t(a.tokens_q) * a.heads)), dim3(256), 0,
                       stream, a, prefix_slots);
    return launch_status();
}

}  // namespace lynx
