// The norms before and after a block, with the gate, the residual and the
// modulation (lynx_block_norm):
//   z  = post(y),  x' = rho x + gate z,  h = pre(x') w + b,  h (1 + scale) + shift
// in one pass over the rows: a row is read once, held in registers as fp32
// through both norms, and x' and h (bf16, or the 8-bit operand) are written
// once.  HBM traffic is what bounds it, at 512 <= C <= 12288.  Two exceptions:
//   - C > 12288 with y: the row, the next row and 32 floats of parameters to a vector do
//     not fit the 256 registers that 8 waves a workgroup leave.  <8, 4> spills 64 of them
//     (fp32 x: 95), and 4096 x 16384 takes 230 us (344) = 2.3 TB/s, 4096 x 12288 94 (138)
//     = 4.3.  <8, 3> with fp32 x spills 10.
//   - Narrow rows: a wave holds one row and one more ahead, so at C = 128 16 of 64 lanes
//     work and few bytes are under way.  With y, 221184 x 128 takes 84 us = 2.7 TB/s, x 256
//     101 = 4.5, 55296 x 512 43 = 5.3.
//
// A workgroup of W waves takes a run of consecutive rows, so that a sample's
// parameters stay in registers from row to row (read anew per row they are as much
// L2 traffic as the row itself), and loads the next row before it works on this
// one.  Lane l of wave w holds channels 8 (64 (i W + w) + l) .. + 7 for i < NV: 512
// channels per wave and i are one scale word of the 8-bit operand, 16 lanes one
// scale.  The parameters are kept as two factors and two terms,
//   x' = rho x + (y - mean) rs a1 + a0,   a1 = post_weight gate, a0 = post_bias gate,
//   h = (x' - mean) rs b1 + b0,   b1 = weight (1 + scale), b0 = bias (1 + scale) + shift.
// Variances are taken around the mean, from the registers.
#include "lynx_fp8.h"

namespace lynx {
namespace {

struct NormArgs {
    const void* x;
    const uint16_t *y, *gate, *post_weight, *post_bias, *weight, *bias, *scale, *shift;
    void* x_out;
    uint16_t* h;
    uint8_t* q;
    uint32_t* q_scale;
    int M, C, rows_per_sample, rows_per_group;
    int64_t gate_stride, scale_stride, shift_stride;
    float rho, post_eps, eps, inv_c;
    int post, norm;
};

struct Vec8 {
    float f[8];
};

__device__ __forceinline__ Vec8 load_bf16(const uint16_t* p) {
    const u32x4 v = *reinterpret_cast<const u32x4*>(p);
    Vec8 r;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r.f[2 * i] = __uint_as_float(v[i] << 16);
        r.f[2 * i + 1] = __uint_as_float(v[i] & 0xFFFF0000u);
    }
    return r;
}

__device__ __forceinline__ void store_bf16(uint16_t* p, const Vec8& v) {
    u32x4 w;
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = uint32_t(__builtin_bit_cast(uint16_t, static_cast<__bf16>(v.f[2 * i]))) |
               (uint32_t(__builtin_bit_cast(uint16_t, static_cast<__bf16>(v.f[2 * i + 1]))) << 16);
    *reinterpret_cast<u32x4*>(p) = w;
}

__device__ __forceinline__ void store_f32(float* p, const Vec8& v) {
    *reinterpret_cast<f32x4*>(p) = f32x4{v.f[0], v.f[1], v.f[2], v.f[3]};
    *reinterpret_cast<f32x4*>(p + 4) = f32x4{v.f[4], v.f[5], v.f[6], v.f[7]};
}

// v plus its copies 8, 4, 2 and 1 lanes round the 16-lane row, from the step `from` on:
// every lane adds the same pairs, so all of them get the same bits
template <int FROM>
__device__ __forceinline__ float row16_sum(float v) {
#define LYNX_ROR(n) \
    if constexpr (n <= FROM) \
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x120 + n, 0xF, 0xF, false))
    LYNX_ROR(8);
    LYNX_ROR(4);
    LYNX_ROR(2);
    LYNX_ROR(1);
#undef LYNX_ROR
    return v;
}

// sum over the row's W waves, in every lane; `slot`: 4 W floats of LDS that no
// earlier sum since the row before last used.  The waves' 16-lane sums are joined by
// every lane from its share of them: fewer instructions than adding them all up.
template <int W>
__device__ __forceinline__ float row_sum(float v, float* slot) {
    v = row16_sum<8>(v);
    if constexpr (W == 1) {
        auto lane = [&](int l) {
            return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l));
        };
        return (lane(0) + lane(16)) + (lane(32) + lane(48));
    } else {
        const int t = threadIdx.x;
        if ((t & 15) == 0) slot[t >> 4] = v;
        __syncthreads();
        if constexpr (W == 8) return row16_sum<8>(slot[t & 15] + slot[16 + (t & 15)]);
        else return row16_sum<2 * W>(slot[t & (4 * W - 1)]);
    }
}

// v becomes v - mean (layer norm); returns 1 / sqrt(mean square + eps), or NaN where the
// sum of squares is not finite: rsqrt(inf) = 0 would turn a row that holds an infinity, or
// squares past fp32's range, into zeros that nobody notices
template <int W, int NV>
__device__ __forceinline__ float normalise(Vec8 (&v)[NV], const bool (&in)[NV], int kind, float inv_c,
                                           float eps, float* slots) {
    if (kind == LYNX_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i].f[j];
        const float mean = row_sum<W>(s, slots) * inv_c;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (in[i]) v[i].f[j] -= mean;  // the others stay 0
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(v[i].f[j], v[i].f[j], s);
    const float sum = row_sum<W>(s, slots + 4 * W);
    return sum < INFINITY ? rsqrtf(fmaf(sum, inv_c, eps)) : __builtin_nanf("");
}

template <int W, int NV, bool XF32, bool HASY>
__global__ __launch_bounds__(64 * W) void block_norm_kernel(const NormArgs A) {
    __shared__ float slots[2][16 * W];
    const int lane = threadIdx.x & 63;
    const int wave = W > 1 ? __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6)) : 0;
    const int begin = int(blockIdx.x) * A.rows_per_group, end = min(begin + A.rows_per_group, A.M);
    int c[NV];
    bool in[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        c[i] = 8 * (64 * (i * W + wave) + lane);
        in[i] = c[i] < A.C;
    }
    struct Row {
        u32x4 x[XF32 ? 2 * NV : NV], y[HASY ? NV : 1];
    };
    auto load = [&](int row, Row& o) {
        const size_t base = size_t(row) * size_t(A.C);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if constexpr (HASY)
                o.y[i] = in[i] ? *reinterpret_cast<const u32x4*>(A.y + base + c[i]) : u32x4{};
            if constexpr (XF32) {
                const float* p = static_cast<const float*>(A.x) + base + c[i];
                o.x[2 * i] = in[i] ? *reinterpret_cast<const u32x4*>(p) : u32x4{};
                o.x[2 * i + 1] = in[i] ? *reinterpret_cast<const u32x4*>(p + 4) : u32x4{};
            } else {
                const uint16_t* p = static_cast<const uint16_t*>(A.x) + base + c[i];
                o.x[i] = in[i] ? *reinterpret_cast<const u32x4*>(p) : u32x4{};
            }
        }
    };
    auto factor = [&](const uint16_t* p, int ch) {  // an absent factor is 1
        if (p) return load_bf16(p + ch);
        return Vec8{{1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f, 1.f}};
    };
    auto term = [&](const uint16_t* p, int ch) { return p ? load_bf16(p + ch) : Vec8{}; };
    struct Params {
        Vec8 a1, a0, b1, b0;
    };
    auto params = [&](int sample, int ch) {
        Params p;
        if constexpr (HASY) {
            p.a1 = factor(A.gate ? A.gate + size_t(sample) * size_t(A.gate_stride) : nullptr, ch);
            p.a0 = term(A.post_bias, ch);
            if (A.post_bias) {  // an absent one stays no term: 0 * inf is NaN
#pragma unroll
                for (int j = 0; j < 8; ++j) p.a0.f[j] *= p.a1.f[j];
            }
            const Vec8 w = factor(A.post_weight, ch);
#pragma unroll
            for (int j = 0; j < 8; ++j) p.a1.f[j] *= w.f[j];
        }
        p.b1 = term(A.scale ? A.scale + size_t(sample) * size_t(A.scale_stride) : nullptr, ch);
        p.b0 = term(A.bias, ch);
        const Vec8 w = factor(A.weight, ch);
        const Vec8 t = term(A.shift ? A.shift + size_t(sample) * size_t(A.shift_stride) : nullptr, ch);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            p.b1.f[j] += 1.f;
            p.b0.f[j] = A.bias ? fmaf(p.b0.f[j], p.b1.f[j], t.f[j]) : t.f[j];
            p.b1.f[j] *= w.f[j];
        }
        return p;
    };

    Row cur;
    load(begin, cur);
    Params kept[NV];
    int sample = -1;
    for (int row = begin; row < end; ++row) {
        const size_t base = size_t(row) * size_t(A.C);
        const int s = row / A.rows_per_sample;
        if (s != sample) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (in[i]) kept[i] = params(s, c[i]);
            sample = s;
        }
        float* sl = slots[row & 1];
        Vec8 v[NV];
        Row next;
        if (row + 1 < end) load(row + 1, next);
        auto widen = [](const u32x4& w) {
            Vec8 r;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                r.f[2 * i] = __uint_as_float(w[i] << 16);
                r.f[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
            }
            return r;
        };
        auto x_of = [&](int i) {
            if constexpr (XF32) {
                Vec8 r;
#pragma unroll
                for (int j = 0; j < 8; ++j) r.f[j] = __uint_as_float(cur.x[2 * i + j / 4][j % 4]);
                return r;
            } else {
                return widen(cur.x[i]);
            }
        };
        if constexpr (HASY) {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = widen(cur.y[i]);
            float rs = 1.f;
            if (A.post) rs = normalise<W>(v, in, A.post, A.inv_c, A.post_eps, sl);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (!in[i]) continue;
                const Params& p = kept[i];
                const Vec8 x = x_of(i);
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    v[i].f[j] = fmaf(A.rho, x.f[j], fmaf(v[i].f[j] * rs, p.a1.f[j], p.a0.f[j]));
                if constexpr (XF32) store_f32(static_cast<float*>(A.x_out) + base + c[i], v[i]);
                else store_bf16(static_cast<uint16_t*>(A.x_out) + base + c[i], v[i]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NV; ++i) v[i] = x_of(i);
        }
        if (A.norm) {
            const float rs = normalise<W>(v, in, A.norm, A.inv_c, A.eps, sl + 8 * W);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                if (in[i]) {
                    const Params& p = kept[i];
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        v[i].f[j] = fmaf(v[i].f[j] * rs, p.b1.f[j], p.b0.f[j]);
                    if (A.h) store_bf16(A.h + base + c[i], v[i]);
                }
                if (A.q) {  // every lane: the group's maximum crosses lanes
                    float m = 0.f;  // keeps a NaN; lanes past C hold zeros
#pragma unroll
                    for (int j = 0; j < 8; ++j)
                        m = __builtin_elementwise_maximum(m, fabsf(v[i].f[j]));
                    const uint32_t byte = fp8_scale_byte(row16_max(__float_as_uint(m)));
                    const float div = fp8_divisor(byte);
                    const float* f = v[i].f;
                    if (in[i])
                        *reinterpret_cast<u32x2*>(A.q + base + c[i]) =
                            u32x2{fp8_pack4(f[0], f[1], f[2], f[3], div),
                                  fp8_pack4(f[4], f[5], f[6], f[7], div)};
                    const int word = i * W + wave;
                    const uint32_t sw = fp8_scale_word(byte);
                    if (lane == 0 && 512 * word < A.C)
                        A.q_scale[size_t(word) * size_t(A.M) + row] = sw;
                }
            }
        }
        cur = next;
    }
}

template <int W, int NV>
void launch(NormArgs& a, bool f32, int cus, hipStream_t s) {
    // at least 16 waves and 4 workgroups a compute unit: enough rows under way to cover
    // the memory's latency, and runs as long as that leaves
    const int groups = cus * (W < 4 ? 16 / W : 4);
    a.rows_per_group = (a.M + groups - 1) / groups;
    const dim3 grid(unsigned((a.M + a.rows_per_group - 1) / a.rows_per_group)), block(64 * W);
    if (a.y) {
        if (f32) hipLaunchKernelGGL((block_norm_kernel<W, NV, true, true>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((block_norm_kernel<W, NV, false, true>), grid, block, 0, s, a);
    } else {
        if (f32) hipLaunchKernelGGL((block_norm_kernel<W, NV, true, false>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((block_norm_kernel<W, NV, false, false>), grid, block, 0, s, a);
    }
}

}  // namespace

lynx_status launch_block_norm(const lynx_norm& d, hipStream_t stream) {
    int cus = 0;
    if (device_cu_count(&cus) != LYNX_OK) return LYNX_ERR_DEVICE;
    NormArgs a;
    a.x = d.x;
    a.y = d.y;
    a.gate = d.gate;
    a.post_weight = d.post_weight;
    a.post_bias = d.post_bias;
    a.weight = d.weight;
    a.bias = d.bias;
    a.scale = d.scale;
    a.shift = d.shift;
    a.x_out = d.x_out;
    a.h = d.h;
    a.q = d.q;
    a.q_scale = reinterpret_cast<uint32_t*>(d.q_scale);
    a.M = int(d.M);
    a.C = int(d.C);
    a.rows_per_sample = int(d.M / d.samples);
    a.gate_stride = d.gate_stride;
    a.scale_stride = d.scale_stride;
    a.shift_stride = d.shift_stride;
    a.rho = d.residual_scale;
    a.post_eps = d.post_eps;
    a.eps = d.eps;
    a.inv_c = 1.f / float(d.C);
    a.post = d.post_norm;
    a.norm = d.norm;
    const bool f32 = d.x_fp32 != 0;
    // As many waves as give each lane 8 channels, up to 8 waves, a power of two: few
    // registers, so many waves to a SIMD.  9216 x 3072 with y and 8-bit output, from HBM:
    // 8 waves 43 us (4.6 TB/s), 4 waves of 16 channels a lane 47, 2 of 24 48; 4096 x 3072
    // with fp32 x and bf16 output 33, 34 and 44.
    const int v = int((d.C + 511) / 512);  // 8-channel vectors of a wave, over the row
    if (v <= 1) launch<1, 1>(a, f32, cus, stream);
    else if (v <= 2) launch<2, 1>(a, f32, cus, stream);
    else if (v <= 4) launch<4, 1>(a, f32, cus, stream);
    else if (v <= 8) launch<8, 1>(a, f32, cus, stream);
    else if (v <= 16) launch<8, 2>(a, f32, cus, stream);
    else if (v <= 24) launch<8, 3>(a, f32, cus, stream);
    else launch<8, 4>(a, f32, cus, stream);
    return launch_status();
}

}  // namespace lynx
