// The norms before and after a block, with the gate, the residual and the
// modulation (lynx_block_norm):
//   z  = post(y),  x' = rho x + gate z,  h = pre(x') w + b,  h (1 + scale) + shift
// in one pass over the rows: a row is read once, held in registers as fp32
// through both norms, and x' and h (bf16, or the 8-bit operand) are written
// once.  HBM traffic is what bounds it.
//
// W waves take a row (1, or 4 for long rows and for few of them); lane l of wave
// w holds channels 8 (64 (i W + w) + l) .. + 7 for i < NV.  512 channels per
// wave and i are one scale word of the 8-bit operand, 16 lanes one scale.
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
    int M, C, rows_per_sample;
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

__device__ __forceinline__ Vec8 load_f32(const float* p) {
    const f32x4 a = *reinterpret_cast<const f32x4*>(p), b = *reinterpret_cast<const f32x4*>(p + 4);
    return Vec8{{a[0], a[1], a[2], a[3], b[0], b[1], b[2], b[3]}};
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

// sum over the row's W waves, in every lane; `slot`: W floats of LDS that no
// earlier sum of the same row used
template <int W>
__device__ __forceinline__ float row_sum(float v, float* slot, int wave) {
#define LYNX_ROR(ctrl) \
    v += __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), ctrl, 0xF, 0xF, false))
    LYNX_ROR(0x128);
    LYNX_ROR(0x124);
    LYNX_ROR(0x122);
    LYNX_ROR(0x121);
#undef LYNX_ROR
    auto lane = [&](int l) { return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), l)); };
    float s = (lane(0) + lane(16)) + (lane(32) + lane(48));
    if constexpr (W > 1) {
        if ((threadIdx.x & 63) == 0) slot[wave] = s;
        __syncthreads();
        s = 0.f;
#pragma unroll
        for (int w = 0; w < W; ++w) s += slot[w];
    }
    return s;
}

// (v - mean) and 1 / sqrt(mean square + eps) of a row; kind 2 is the layer norm
template <int W, int NV>
__device__ __forceinline__ float normalise(Vec8 (&v)[NV], const bool (&in)[NV], int kind, float inv_c,
                                           float eps, float* slots, int wave) {
    if (kind == LYNX_NORM_LAYER) {
        float s = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) s += v[i].f[j];
        const float mean = row_sum<W>(s, slots, wave) * inv_c;
#pragma unroll
        for (int i = 0; i < NV; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i].f[j] = in[i] ? v[i].f[j] - mean : 0.f;
    }
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) s = fmaf(v[i].f[j], v[i].f[j], s);
    return rsqrtf(fmaf(row_sum<W>(s, slots + W, wave), inv_c, eps));
}

template <int W, int NV, bool XF32>
__global__ __launch_bounds__(256) void block_norm_kernel(const NormArgs A) {
    __shared__ float slots[4 * W];
    const int lane = threadIdx.x & 63;
    const int wid = __builtin_amdgcn_readfirstlane(int(threadIdx.x >> 6));
    const int wave = W > 1 ? wid : 0;
    const int row = W > 1 ? int(blockIdx.x) : int(blockIdx.x) * 4 + wid;
    if (row >= A.M) return;
    const int sample = row / A.rows_per_sample;
    const size_t base = size_t(row) * size_t(A.C);
    int c[NV];
    bool in[NV];
    Vec8 v[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        c[i] = 8 * (64 * (i * W + wave) + lane);
        in[i] = c[i] < A.C;
    }
    auto load_x = [&](int i) {
        if constexpr (XF32) return load_f32(static_cast<const float*>(A.x) + base + c[i]);
        else return load_bf16(static_cast<const uint16_t*>(A.x) + base + c[i]);
    };
    if (A.y) {
        Vec8 x[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = in[i] ? load_bf16(A.y + base + c[i]) : Vec8{};
#pragma unroll
        for (int i = 0; i < NV; ++i) x[i] = in[i] ? load_x(i) : Vec8{};
        float rs = 1.f;
        if (A.post) rs = normalise<W>(v, in, A.post, A.inv_c, A.post_eps, slots, wave);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (!in[i]) continue;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i].f[j] *= rs;
            if (A.post_weight) {
                const Vec8 p = load_bf16(A.post_weight + c[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i].f[j] *= p.f[j];
            }
            if (A.post_bias) {
                const Vec8 p = load_bf16(A.post_bias + c[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i].f[j] += p.f[j];
            }
            if (A.gate) {
                const Vec8 p = load_bf16(A.gate + size_t(sample) * size_t(A.gate_stride) + c[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i].f[j] *= p.f[j];
            }
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i].f[j] = fmaf(A.rho, x[i].f[j], v[i].f[j]);
            if constexpr (XF32) store_f32(static_cast<float*>(A.x_out) + base + c[i], v[i]);
            else store_bf16(static_cast<uint16_t*>(A.x_out) + base + c[i], v[i]);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) v[i] = in[i] ? load_x(i) : Vec8{};
    }
    if (!A.norm) return;

    const float rs = normalise<W>(v, in, A.norm, A.inv_c, A.eps, slots + 2 * W, wave);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        if (in[i]) {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[i].f[j] *= rs;
            if (A.weight) {
                const Vec8 p = load_bf16(A.weight + c[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i].f[j] *= p.f[j];
            }
            if (A.bias) {
                const Vec8 p = load_bf16(A.bias + c[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i].f[j] += p.f[j];
            }
            if (A.scale) {
                const Vec8 p = load_bf16(A.scale + size_t(sample) * size_t(A.scale_stride) + c[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i].f[j] *= 1.f + p.f[j];
            }
            if (A.shift) {
                const Vec8 p = load_bf16(A.shift + size_t(sample) * size_t(A.shift_stride) + c[i]);
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i].f[j] += p.f[j];
            }
            if (A.h) store_bf16(A.h + base + c[i], v[i]);
        }
        if (A.q) {  // every lane: the group's maximum crosses lanes
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j)
                m = max(m, in[i] ? __float_as_uint(v[i].f[j]) & 0x7FFFFFFFu : 0u);
            const uint32_t byte = fp8_scale_byte(row16_max(m));
            const float div = fp8_divisor(byte);
            const float* f = v[i].f;
            if (in[i])
                *reinterpret_cast<u32x2*>(A.q + base + c[i]) =
                    u32x2{fp8_pack4(f[0], f[1], f[2], f[3], div), fp8_pack4(f[4], f[5], f[6], f[7], div)};
            const int word = i * W + wave;
            const uint32_t sw = fp8_scale_word(byte);
            if (lane == 0 && 512 * word < A.C) A.q_scale[size_t(word) * size_t(A.M) + row] = sw;
        }
    }
}

template <int W, int NV>
void launch(const NormArgs& a, bool f32, hipStream_t s) {
    const dim3 grid(unsigned(W > 1 ? a.M : (a.M + 3) / 4));
    if (f32) hipLaunchKernelGGL((block_norm_kernel<W, NV, true>), grid, dim3(256), 0, s, a);
    else hipLaunchKernelGGL((block_norm_kernel<W, NV, false>), grid, dim3(256), 0, s, a);
}

template <int W>
void launch_nv(const NormArgs& a, bool f32, hipStream_t s) {
    const int nv = (a.C + 512 * W - 1) / (512 * W);  // <= 8
    if (nv <= 1) launch<W, 1>(a, f32, s);
    else if (nv <= 2) launch<W, 2>(a, f32, s);
    else if (nv <= 4) launch<W, 4>(a, f32, s);
    else if (nv <= 6) launch<W, 6>(a, f32, s);
    else launch<W, 8>(a, f32, s);
}

}  // namespace

lynx_status launch_block_norm(const lynx_norm& d, hipStream_t stream) {
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
    if (d.C > 4096 || (d.C > 512 && d.M < 2048)) launch_nv<4>(a, d.x_fp32 != 0, stream);
    else launch_nv<1>(a, d.x_fp32 != 0, stream);
    return launch_status();
}

}  // namespace lynx
