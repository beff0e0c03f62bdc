// Rotary positions of q and k with the norm of each head before (lynx_qk_rotary):
//   x <- x rsqrt(mean x^2 + eps) w,   (x_m, x_n) <- (x_m cos - x_n sin, x_m sin + x_n cos)
// HBM traffic is what bounds it: every row (a token's head) is read and written once.  20000 x 32 x
// 128 without a norm 62 us (5.3 TB/s, a copy's rate); 8191 x 32 x 72 with norm 21.6 (3.5).
//
// A row is held by D / 8 lanes, 8 channels each; a wave holds 64 / (D / 8) rows side by side, all
// heads of one token (of several tokens where there are few heads), and goes through the
// token's heads U such groups at a time (two: 22.9 us; three 25.7, four 26.4, since fewer waves
// fit).  Angles cost fp64 arithmetic, so they are taken once a
// token: the wave's lanes compute the cosines and sines of its pairs while the first rows are
// under way, and each lane keeps those of its 8 channels for all heads.  The angle is taken in
// turns, t = position * (frequency / 2 pi), which is off by 2^-52 of itself at most (2^-23.6 of a
// turn at position 2^31), and t - rint(t) is exact, before it is rounded to fp32 (2^-26).
//
// A pair's other channel is the lane's own (adjacent pairs) or lies R / 2 further: such rows cross
// lanes through LDS, as bf16 words.  The norm's weights go into the factors:
//   y_j = rsqrt(..) (x_j (w_j cos) + other_j (w_other sin)),
// kept for q's heads, then for k's: a group of rows holds heads of one of them.
#include <algorithm>
#include <cmath>
#include <type_traits>

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
    int tokens, q_heads, heads, D;      // heads: q's and k's together
    int lanes, side, per_wave;          // lanes of a row; rows side by side; tokens of a wave
    int q_groups, groups, split;        // groups of `side` heads: q's, all, of a wave
    int axes, pairs, positions_fp32, norm;
    float eps, inv_d;
    int first[4];              // each axis' first pair (pairs, where there is no axis)
    double turns[kMaxPairs];   // a pair's frequency over 2 pi
};

// Sum over the lanes of a row, in all of them; `part`: kParts floats of LDS of the wave's own, zero
// where no lane writes.
constexpr int kParts = 128;  // (64 / lanes + 1) rows of `pad` floats, the last one of lanes that are left over
__device__ __forceinline__ float row_total(float s, int lanes, int place, int in_row, float* part) {
    auto ror = [&](auto n) {
        return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(s), 0x120 + n(), 0xF, 0xF, false));
    };
    auto by = [](auto n) { return n; };
    if (lanes == 16) {
        s += ror(by(std::integral_constant<int, 8>{}));
        s += ror(by(std::integral_constant<int, 4>{}));
        s += ror(by(std::integral_constant<int, 2>{}));
        s += ror(by(std::integral_constant<int, 1>{}));
        return s;
    }
    if ((lanes & (lanes - 1)) == 0) {
        for (int d = 1; d < lanes; d *= 2) s += __shfl_xor(s, d);
        return s;
    }
    // rows of 3, 5 .. 7, 9 .. 15, 17 .. 31 lanes: their parts side by side, the rest zero
    const int pad = lanes < 4 ? 4 : lanes < 8 ? 8 : lanes < 16 ? 16 : 32;
    float* mine = part + place * pad;
    mine[in_row] = s;
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    auto add = [&](int from, int to) {
        f32x4 v = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int i = from; i < to; i += 4) v += *reinterpret_cast<const f32x4*>(mine + i);
        return (v[0] + v[1]) + (v[2] + v[3]);
    };
    s = pad == 4 ? add(0, 4) : pad == 8 ? add(0, 8) : add(0, 16);
    if (pad == 32) s += add(16, 32);
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
    __builtin_amdgcn_wave_barrier();
    return s;
}

// HALVES: 0 adjacent pairs; 1 pairs R / 2 apart, a multiple of 8; 2 any R / 2
template <int U, int HALVES>
__global__ __launch_bounds__(256) void rotary_kernel(const RotaryArgs A) {
    __shared__ __attribute__((aligned(16))) float2 table[4][256];  // cosine and sine
    __shared__ u32x4 swap[4][HALVES ? 64 : 1];
    __shared__ __attribute__((aligned(16))) float part[4][kParts];
    const int lane = threadIdx.x & 63, wave = sgpr(int(threadIdx.x >> 6));
    const int item = int(blockIdx.x) * 4 + wave;
    const int waves = (A.groups + A.split - 1) / A.split;  // of a token
    const int set = sgpr(item / waves), t0 = set * A.per_wave;
    if (t0 >= A.tokens) return;
    const int begin = (item - set * waves) * A.split, end = min(begin + A.split, A.groups);
    const int place = lane / A.lanes, in_row = lane - place * A.lanes, ch = 8 * in_row;
    // This lane's token, and its first head.  Few heads: the wave holds several tokens, and each
    // lane one head, of q or of k.
    const bool few = A.per_wave > 1;
    const int dt = few ? place / A.heads : 0, first = few ? place - dt * A.heads : place;
    const int64_t t = t0 + dt;
    const bool there = place < A.side && dt < A.per_wave && t < A.tokens;

    // Channel m's other one, and whether it is the first of the two
    const int half = A.pairs;
    auto other = [&](int m) {
        if constexpr (HALVES == 0) return m ^ 1;
        return m >= 2 * half ? m : m < half ? m + half : m - half;
    };
    const int och = HALVES == 1 ? other(ch) : ch;

    if (A.norm && (A.lanes & (A.lanes - 1)) != 0)
        for (int i = lane; i < kParts; i += 64) part[wave][i] = 0.f;

    u32x4 x[U];
    // rows of groups g .. g + U - 1: those of one of q and k
    struct Rows {
        const uint16_t* in;
        uint16_t* out;
        int64_t step, out_step;
        int heads;
        bool q;
    };
    auto rows = [&](bool q, int head) {
        Rows r;
        r.q = q;
        r.in = q ? A.q + t * A.q_stride + head * A.q_head_stride : A.k + t * A.k_stride + head * A.k_head_stride;
        r.out = q ? A.q_out + t * A.q_out_stride + head * A.q_out_head_stride
                  : A.k_out + t * A.k_out_stride + head * A.k_out_head_stride;
        r.in += ch;
        r.out += ch;
        r.step = A.side * (q ? A.q_head_stride : A.k_head_stride);
        r.out_step = A.side * (q ? A.q_out_head_stride : A.k_out_head_stride);
        r.heads = there ? (q ? A.q_heads : A.heads - A.q_heads) - head : 0;
        return r;
    };
    // group g0 of a part is its group 0; g1: where the wave's groups of it end
    auto load = [&](const Rows& r, int g, int g1) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            x[u] = u32x4{};
            if (g + u < g1 && (g + u) * A.side < r.heads)
                x[u] = *reinterpret_cast<const u32x4*>(r.in + (g + u) * r.step);
        }
    };
    const int qe = min(end, A.q_groups);
    Rows cur = few ? rows(first < A.q_heads, first < A.q_heads ? first : first - A.q_heads) : rows(begin < qe, first);
    int g = few || begin < qe ? begin : begin - A.q_groups, g1 = few || begin < qe ? qe : end - A.q_groups;
    load(cur, g, g1);

    for (int e = lane; e < A.per_wave * half; e += 64) {
        const int d = e / half, p = e - d * half;
        const int axis = (p >= A.first[1]) + (p >= A.first[2]) + (p >= A.first[3]);
        const int64_t i = int64_t(min(t0 + d, A.tokens - 1)) * A.axes + axis;
        const double pos = A.positions_fp32 ? double(static_cast<const float*>(A.positions)[i])
                                            : double(static_cast<const int*>(A.positions)[i]);
        const double turn = pos * A.turns[p];
        float s, c;
        sincospif(2.f * float(turn - rint(turn)), &s, &c);
        table[wave][e] = float2{c, s};
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_wave_barrier();

    auto widen = [](const u32x4& v, float (&f)[8]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(v[i] << 16);
            f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
        }
    };
    for (;;) {
        // this part's factors
        float c[8], s[8];
        const uint16_t* weight = cur.q ? A.q_weight : A.k_weight;
        if (!there) weight = nullptr;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            const int m = ch + j, o = other(m);
            const int p = HALVES ? (m < half ? m : m - half) : m / 2;
            const float2 cs = table[wave][min(dt * half + min(p, half - 1), 255)];
            const bool low = HALVES ? m < half : (j & 1) == 0;
            c[j] = m < 2 * half ? cs.x : 1.f;
            s[j] = m < 2 * half ? (low ? -cs.y : cs.y) : 0.f;
            if (HALVES == 2 && weight && m < 2 * half) s[j] *= __uint_as_float(uint32_t(weight[o]) << 16);
        }
        if (weight) {
            float w[8], ow[8];
            widen(*reinterpret_cast<const u32x4*>(weight + ch), w);
            if constexpr (HALVES == 1) widen(*reinterpret_cast<const u32x4*>(weight + och), ow);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                c[j] *= w[j];
                if constexpr (HALVES == 0) s[j] *= w[j ^ 1];
                if constexpr (HALVES == 1) s[j] *= ow[j];
            }
        }
        for (; g < g1; g += U) {
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float v[8], o[8], r[8];
                widen(x[u], v);
                if constexpr (HALVES) {
                    swap[wave][lane] = x[u];
                    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                    if constexpr (HALVES == 1) {
                        widen(swap[wave][min(lane - in_row + och / 8, 63)], o);
                    } else {
                        const uint16_t* words = reinterpret_cast<const uint16_t*>(swap[wave]);
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            o[j] = __uint_as_float(uint32_t(words[min((lane - in_row) * 8 + other(ch + j), 511)]) << 16);
                    }
                    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
                    __builtin_amdgcn_wave_barrier();
                } else {
#pragma unroll
                    for (int j = 0; j < 8; ++j) o[j] = v[j ^ 1];
                }
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = fmaf(o[j], s[j], v[j] * c[j]);
                if (2 * half < A.D) {  // not turned: the other's product is no term (it may be NaN)
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        if (ch + j >= 2 * half) r[j] = v[j] * c[j];
                }
                if (A.norm) {
                    float q = 0.f;
#pragma unroll
                    for (int j = 0; j < 8; ++j) q = fmaf(v[j], v[j], q);
                    q = row_total(q, A.lanes, place, in_row, part[wave]);
                    const float rs = q < INFINITY ? rsqrtf(fmaf(q, A.inv_d, A.eps)) : __builtin_nanf("");
#pragma unroll
                    for (int j = 0; j < 8; ++j) r[j] *= rs;
                }
                if (g + u < g1 && (g + u) * A.side < cur.heads) {
                    u32x4 y;
#pragma unroll
                    for (int i = 0; i < 4; ++i) y[i] = pack_bf16(r[2 * i], r[2 * i + 1]);
                    *reinterpret_cast<u32x4*>(cur.out + (g + u) * cur.out_step) = y;
                }
            }
            if (g + U < g1) load(cur, g + U, g1);
        }
        if (few || end <= A.q_groups || !cur.q) break;
        cur = rows(false, first);
        g = 0;
        g1 = end - A.q_groups;
        load(cur, g, g1);
    }
}

template <int U>
void launch_rotary(const RotaryArgs& a, int halves, hipStream_t s) {
    const int64_t waves = (int64_t(a.tokens) + a.per_wave - 1) / a.per_wave * ((a.groups + a.split - 1) / a.split);
    const dim3 grid(unsigned((waves + 3) / 4));
    if (halves == 0) hipLaunchKernelGGL((rotary_kernel<U, 0>), grid, dim3(256), 0, s, a);
    else if (halves == 1) hipLaunchKernelGGL((rotary_kernel<U, 1>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((rotary_kernel<U, 2>), grid, dim3(256), 0, s, a);
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
    a.D = int(d.head_dim);
    a.lanes = a.D / 8;
    a.side = 64 / a.lanes;
    a.per_wave = a.heads < a.side ? a.side / a.heads : 1;
    a.q_groups = a.per_wave > 1 ? 1 : (a.q_heads + a.side - 1) / a.side;
    a.groups = a.q_groups + (a.per_wave > 1 ? 0 : (int(d.k_heads) + a.side - 1) / a.side);
    a.axes = d.axes;
    a.positions_fp32 = d.positions_fp32;
    a.norm = d.norm == LYNX_NORM_RMS;
    a.eps = d.eps;
    a.inv_d = 1.f / float(d.head_dim);
    int R = 0;
    for (int i = 0; i < d.axes; ++i) R += d.axis_dims[i];
    a.pairs = R / 2;
    const long double log2_theta = std::log2(static_cast<long double>(d.theta));  // (pow takes 0.5 us an axis)
    for (int i = 0, p = 0; i < 4; ++i) {
        a.first[i] = i < d.axes ? p : a.pairs;
        if (i >= d.axes) continue;
        // theta^(-2 j / n) as powers of theta^(-2 / n), in 64 bits of fraction, so that 128 products
        // leave one rounding to 53 bits: in those they were off by 2^-21.9 of a turn at position 2^31
        const bool joint = d.ladder == LYNX_LADDER_JOINT;
        const long double step = std::exp2(-2.0L / (joint ? R : d.axis_dims[i]) * log2_theta);
        long double f = 0.159154943091895335768883763372514362L;  // 1 / 2 pi
        if (joint)
            for (int j = 0; j < p; ++j) f *= step;
        for (int j = 0; j < d.axis_dims[i] / 2; ++j, f *= step) a.turns[p++] = double(f);
    }
    const int halves = d.pairs == LYNX_PAIRS_ADJACENT ? 0 : a.pairs % 8 == 0 ? 1 : 2;
    // A token's groups go to several waves while there are fewer than three to a SIMD: what a wave
    // does before its rows (positions, angles, weights) costs as much as some rows.  4608 x 48 x
    // 128: all 12 groups to a wave 22.9 us (4.95 TB/s), 6 24.9, 3 26.1.
    const int64_t want = 256 * 12, sets = (int64_t(a.tokens) + a.per_wave - 1) / a.per_wave;
    const int64_t parts = std::min<int64_t>(a.groups, (want + sets - 1) / sets);
    a.split = int((a.groups + parts - 1) / parts);
    if (a.split <= 1) launch_rotary<1>(a, halves, stream);
    else launch_rotary<2>(a, halves, stream);
    return launch_status();
}

}  // namespace lynx
