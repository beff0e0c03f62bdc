// Joins the partial results of a row's chunks of keys (lynx_attention):
//   M = max m_i,   o = sum 2^(m_i - M) o_i / sum 2^(m_i - M) l_i,   lse = (M + log2 l) ln 2 (l of
// unrounded weights).  The partial results' bytes bound it.  A row's slots are weighed by its
// lanes side by side, then 32 lanes take 4 channels each; a workgroup of 256 threads takes 8 rows
// of one such group, or, where there are many slots, fewer rows and the slots dealt to the groups:
// 1024 rows of up to 17 slots 5.5 us, of which 4 are a launch's own.
#include "lynx_attn.h"

namespace lynx {
namespace {

template <int GROUPS>  // of 32 lanes to a row
__global__ __launch_bounds__(256) void attn_join_kernel(const AttnArgs A, int prefix_slots) {
    constexpr int ROWS = 8 / GROUPS, SLOTS = 2 * kMaxChunks;
    __shared__ float f[ROWS][SLOTS];
    __shared__ f32x4 sum[8][32];
    const int lane = threadIdx.x & 31, group = int(threadIdx.x >> 5) % GROUPS, r = int(threadIdx.x >> 5) / GROUPS;
    const int64_t rows = int64_t(A.tokens_q) * A.heads, row = int64_t(blockIdx.x) * ROWS + r;
    const int token = int(row / A.heads), head = int(row - int64_t(token) * A.heads);
    bool work = row < rows;
    if (work && A.cu_q)  // rows of no sequence
        work = token >= A.cu_q[0] && token < A.cu_q[A.batch];
    int n = 0;
    if (work) n = prefix_slots + clampi(A.part_n[row], 1, A.slots - prefix_slots);
    if (n == 1 && !A.force_part) n = 0;  // written already
    const int64_t first = row * A.slots;
    // weights of the slots, by every group of the row alike
    float M = -INFINITY, l = 0.f, le = 0.f;
    float4 ml[SLOTS / 32];
#pragma unroll
    for (int i = 0; i < SLOTS / 32; ++i) {
        ml[i] = float4{-INFINITY, 0.f, 0.f, 0.f};
        if (lane + 32 * i < n) ml[i] = A.part_ml[first + lane + 32 * i];
        M = fmaxf(M, ml[i].x);
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) M = fmaxf(M, __shfl_xor(M, d));
#pragma unroll
    for (int i = 0; i < SLOTS / 32; ++i) {
        // no key was seen: nothing to scale
        const float w = ml[i].x == -INFINITY ? 0.f : __builtin_amdgcn_exp2f(ml[i].x - M);
        l += w * ml[i].y;
        le += w * ml[i].z;
        if (group == 0) f[r][lane + 32 * i] = w;
    }
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
        l += __shfl_xor(l, d);
        le += __shfl_xor(le, d);
    }
    __syncthreads();
    const int c = 4 * lane;
    const bool in = c < A.D;
    f32x4 o = {0.f, 0.f, 0.f, 0.f};
    const float* p = A.part_o + first * A.D + c;
#pragma unroll 4
    for (int i = group; i < n; i += GROUPS) {
        const float w = f[r][i];
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
        if (in) v = *reinterpret_cast<const f32x4*>(p + int64_t(i) * A.D);
#pragma unroll
        for (int e = 0; e < 4; ++e) o[e] = fmaf(w, v[e], o[e]);
    }
    if constexpr (GROUPS > 1) {
        sum[threadIdx.x >> 5][lane] = o;
        __syncthreads();
        if (group != 0) return;
#pragma unroll
        for (int i = 1; i < GROUPS; ++i)
#pragma unroll
            for (int e = 0; e < 4; ++e) o[e] += sum[r * GROUPS + i][lane][e];
    }
    if (n == 0) return;
    const float inv = l == 0.f ? 0.f : 1.f / l;
    if (in) {
        const int b = A.addr_len == 0 ? 0 : token / A.addr_len;
        uint16_t* out = A.out + b * A.o_b + (token - b * A.addr_len) * A.o_t + head * A.o_h + c;
        *reinterpret_cast<u32x2*>(out) = u32x2{pack_bf16(o[0] * inv, o[1] * inv), pack_bf16(o[2] * inv, o[3] * inv)};
    }
    if (A.lse && lane == 0) A.lse[row] = le == 0.f ? -INFINITY : (M + log2f(le)) * kLn2;
}

}  // namespace

lynx_status launch_attn_join(const AttnArgs& a, int prefix_slots, hipStream_t stream) {
    // workgroups for every unit, and not many more
    const int64_t rows = int64_t(a.tokens_q) * a.heads;
    if (a.slots <= 4 || rows > 4096)
        hipLaunchKernelGGL((attn_join_kernel<1>), dim3(unsigned((rows + 7) / 8)), dim3(256), 0, stream, a,
                           prefix_slots);
    else if (a.slots <= 16 || rows > 1024)
        hipLaunchKernelGGL((attn_join_kernel<4>), dim3(unsigned((rows + 1) / 2)), dim3(256), 0, stream, a,
                           prefix_slots);
    else
        hipLaunchKernelGGL((attn_join_kernel<8>), dim3(unsigned(rows)), dim3(256), 0, stream, a, prefix_slots);
    return launch_status();
}

}  // namespace lynx
