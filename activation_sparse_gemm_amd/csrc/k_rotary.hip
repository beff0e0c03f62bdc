// Rotary positions of q and k with the norm of each head before (lynx_qk_rotary):
//   x <- x rsqrt(mean x^2 + eps) w,   (x_m, x_n) <- (x_m cos - x_n sin, x_m sin + x_n cos)
// HBM traffic is what bounds it: every row (a token's head) is read and written once.
//
// A row is held by LPR lanes, 8 channels each.  A workgroup takes a run of rows in the order
// token, head (q's heads, then k's), loads all of them, and computes the cosines and sines
// of the tokens that its rows belong to once, into LDS, while the loads are under way:
// angles cost fp64 arithmetic, but once a token and not once a head.  The angle is taken in
// turns, t = position * (frequency / 2 pi), in fp64, and t - rint(t) is exact, so positions
// far from the start lose nothing.
//
// A pair's other channel is the lane's own neighbour (adjacent pairs) or lies R / 2 further:
// such rows cross lanes through LDS, as bf16 words.
#include <cmath>

#include "lynx_attn.h"

namespace lynx {
namespace {

constexpr int kMaxPairs = 128;

struct RotaryArgs {
    const uint16_t *q, *k, *q_weight, *k_weight;
    const void* positions;
    uint16_t *q_out, *k_out;
    int64_t q_stride, q_head_stride, k_stride, k_head_stride;
    int64_t q_out_stride, q_out_head_stride, k_out_stride, k_out_head_stride;
    int tokens, q_heads, heads, D, rows;  // heads, rows: q's and k's together
    int axes, pairs, positions_fp32, halves, norm;
    float eps, inv_d;
    int first[4];              // each axis' first pair (pairs, where there is no axis)
    double turns[kMaxPairs];   // a pair's frequency over 2 pi
};

struct Row8 {
    float f[8];
};

__device__ __forceinline__ Row8 widen8(const u32x4& w) {
    Row8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.f[2 * i] = __uint_as_float(w[i] << 16);
        r.f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    return r;
}

// U rows a lane; LPR lanes (a power of two) a row
template <int LPR, int U, bool HALVES>
__global__ __launch_bounds__(256) void rotary_kernel(const RotaryArgs A) {
    constexpr int RPS = 256 / LPR;          // rows side by side in a workgroup
    constexpr int ROWS = RPS * U;
    extern __shared__ __attribute__((aligned(16))) char smem[];
    float2* cs = reinterpret_cast<float2*>(smem);  // [tokens of the workgroup][pairs]
    __shared__ u32x4 swap[HALVES ? 256 : 1];
    const int tid = threadIdx.x, lane = tid % LPR, slot = tid / LPR;
    const int begin = int(blockIdx.x) * ROWS, end = min(begin + ROWS, A.rows);
    const int token0 = begin / A.heads, tokens = (end - 1) / A.heads - token0 + 1;
    const int ch = 8 * lane;
    const bool in = ch < A.D;

    u32x4 x[U];
    int64_t at[U];
    int tok[U];
    bool isq[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int row = min(begin + u * RPS + slot, end - 1);
        const int t = row / A.heads, h = row - t * A.heads;
        tok[u] = t;
        isq[u] = h < A.q_heads;
        const int hk = h - A.q_heads;
        const uint16_t* p = isq[u] ? A.q + t * A.q_stride + h * A.q_head_stride
                                   : A.k + t * A.k_stride + hk * A.k_head_stride;
        at[u] = isq[u] ? t * A.q_out_stride + h * A.q_out_head_stride
                       : t * A.k_out_stride + hk * A.k_out_head_stride;
        x[u] = in ? *reinterpret_cast<const u32x4*>(p + ch) : u32x4{};
    }
    u32x4 wq = {}, wk = {};
    if (A.q_weight && in) wq = *reinterpret_cast<const u32x4*>(A.q_weight + ch);
    if (A.k_weight && in) wk = *reinterpret_cast<const u32x4*>(A.k_weight + ch);

    for (int e = tid; e < tokens * A.pairs; e += 256) {
        const int t = e / A.pairs, p = e - t * A.pairs;
        const int axis = (p >= A.first[1]) + (p >= A.first[2]) + (p >= A.first[3]);
        const size_t i = size_t(token0 + t) * size_t(A.axes) + size_t(axis);
        const double pos = A.positions_fp32 ? double(static_cast<const float*>(A.positions)[i])
                                            : double(static_cast<const int*>(A.positions)[i]);
        const double turn = pos * A.turns[p];
        float s, c;
        sincospif(2.f * float(turn - rint(turn)), &s, &c);
        cs[e] = float2{c, s};
    }
    __syncthreads();

    const int half = A.pairs;
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const int row = begin + u * RPS + slot;
        Row8 v = widen8(x[u]);
        float rs = 1.f;
        if (A.norm) {
            float s = 0.f;
#pragma unroll
            for (int j = 0; j < 8; ++j) s = fmaf(v.f[j], v.f[j], s);
#pragma unroll
            for (int d = 1; d < LPR; d *= 2) s += __shfl_xor(s, d);
            rs = s < INFINITY ? rsqrtf(fmaf(s, A.inv_d, A.eps)) : __builtin_nanf("");
        }
        const float2* c = cs + (tok[u] - token0) * A.pairs;
        const uint16_t* weight = isq[u] ? A.q_weight : A.k_weight;
        const Row8 w = widen8(isq[u] ? wq : wk);
        if (weight) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v.f[j] *= rs * w.f[j];
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v.f[j] *= rs;
        }
        if constexpr (!HALVES) {
#pragma unroll
            for (int j = 0; j < 8; j += 2) {
                const int p = (ch + j) / 2;
                if (p < half) {
                    const float a = v.f[j], b = v.f[j + 1];
                    v.f[j] = a * c[p].x - b * c[p].y;
                    v.f[j + 1] = a * c[p].y + b * c[p].x;
                }
            }
        } else {
            // the row crosses lanes through this wave's part of `swap` alone
            swap[tid] = x[u];
            __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
            __builtin_amdgcn_wave_barrier();
            const uint16_t* words = reinterpret_cast<const uint16_t*>(swap + tid - lane);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                const int m = ch + j;
                if (m < 2 * half) {
                    const bool low = m < half;
                    const int n = low ? m + half : m - half, p = low ? m : n;
                    float o = __uint_as_float(uint32_t(words[n]) << 16);
                    o *= weight ? rs * __uint_as_float(uint32_t(weight[n]) << 16) : rs;
                    v.f[j] = low ? v.f[j] * c[p].x - o * c[p].y : o * c[p].y + v.f[j] * c[p].x;
                }
            }
            __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
            __builtin_amdgcn_wave_barrier();
        }
        if (in && row < end) {
            u32x4 o;
#pragma unroll
            for (int i = 0; i < 4; ++i) o[i] = pack_bf16(v.f[2 * i], v.f[2 * i + 1]);
            *reinterpret_cast<u32x4*>((isq[u] ? A.q_out : A.k_out) + at[u] + ch) = o;
        }
    }
}

template <int LPR, int U>
void launch_rotary(const RotaryArgs& a, hipStream_t s) {
    constexpr int ROWS = 256 / LPR * U;
    const dim3 grid(unsigned((int64_t(a.rows) + ROWS - 1) / ROWS));
    const int tokens = min((ROWS - 1 + a.heads - 1) / a.heads + 1, ROWS);  // that a run can touch
    const size_t lds = size_t(tokens) * size_t(a.pairs) * sizeof(float2);
    if (a.halves) hipLaunchKernelGGL((rotary_kernel<LPR, U, true>), grid, dim3(256), lds, s, a);
    else hipLaunchKernelGGL((rotary_kernel<LPR, U, false>), grid, dim3(256), lds, s, a);
}

}  // namespace

lynx_status launch_qk_rotary(const lynx_rotary& d, hipStream_t stream) {
    RotaryArgs a = {};
    a.q = d.q;
    a.k = d.k;
    a.q_weight = d.q_weight;
    a.k_weight = d.k_weight;
    a.positions = d.positions;
    a.q_out = d.q_out;
    a.k_out = d.k_out;
    a.q_stride = d.q_stride;
    a.q_head_stride = d.q_head_stride;
    a.k_stride = d.k_stride;
    a.k_head_stride = d.k_head_stride;
    a.q_out_stride = d.q_out_stride;
    a.q_out_head_stride = d.q_out_head_stride;
    a.k_out_stride = d.k_out_stride;
    a.k_out_head_stride = d.k_out_head_stride;
    a.tokens = int(d.tokens);
    a.q_heads = int(d.q_heads);
    a.heads = int(d.q_heads + d.k_heads);
    a.rows = a.tokens * a.heads;
    a.D = int(d.head_dim);
    a.axes = d.axes;
    a.positions_fp32 = d.positions_fp32;
    a.halves = d.pairs == LYNX_PAIRS_HALVES;
    a.norm = d.norm == LYNX_NORM_RMS;
    a.eps = d.eps;
    a.inv_d = 1.f / float(d.head_dim);
    int R = 0;
    for (int i = 0; i < d.axes; ++i) R += d.axis_dims[i];
    a.pairs = R / 2;
    for (int i = 0, p = 0; i < 4; ++i) {
        a.first[i] = i < d.axes ? p : a.pairs;
        if (i >= d.axes) continue;
        // theta^(-2 j / n) as powers of theta^(-2 / n): 128 roundings of 2^-53 at most
        const bool joint = d.ladder == LYNX_LADDER_JOINT;
        const double step = std::pow(d.theta, -2.0 / (joint ? R : d.axis_dims[i]));
        double f = 0.15915494309189535;  // 1 / 2 pi
        if (joint)
            for (int j = 0; j < p; ++j) f *= step;
        for (int j = 0; j < d.axis_dims[i] / 2; ++j, f *= step) a.turns[p++] = f;
    }
    const int lanes = (a.D + 7) / 8;
    if (lanes <= 4) launch_rotary<4, 1>(a, stream);
    else if (lanes <= 8) launch_rotary<8, 1>(a, stream);
    else if (lanes <= 16) launch_rotary<16, 1>(a, stream);
    else launch_rotary<32, 1>(a, stream);
    return launch_status();
}

}  // namespace lynx
