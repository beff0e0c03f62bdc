// Internal declarations of the 8-bit path: the operand layout, the device
// helpers that quantise, and the launchers (validated arguments only).
#pragma once

#include "lynx_internal.h"

namespace lynx {

typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kFp8Block = 128;        // channels (and weight rows) per scale
constexpr uint32_t kScaleOne = 127;   // E8M0 byte of 1
constexpr uint32_t kScaleNaN = 255;   // E8M0 byte of NaN

// Scale words of a row: four K blocks to a 32-bit word.
inline __host__ __device__ int fp8_scale_words(int K) { return (K + 511) / 512; }

// max over the 16 lanes of a DPP row, in every lane of the row
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x128, 0xF, 0xF, false)));
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x124, 0xF, 0xF, false)));
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x122, 0xF, 0xF, false)));
    v = max(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), 0x121, 0xF, 0xF, false)));
    return v;
}

// E8M0 byte for a group whose largest magnitude has the fp32 bits `amax`: the
// smallest power of two 2^e with amax <= 448 2^e.  448 = 7/8 2^9, so with
// amax = f 2^x (f in [1/2, 1)) e = x - 9, or x - 8 where f > 7/8.  Magnitudes
// are compared as integers, so that a NaN (above every number) is not lost.
__device__ __forceinline__ uint32_t fp8_scale_byte(uint32_t amax) {
    const float a = __uint_as_float(amax);
    int e = __builtin_amdgcn_frexp_expf(a) - (__builtin_amdgcn_frexp_mantf(a) > 0.875f ? 8 : 9);
    e = max(e, -127);
    const uint32_t b = amax == 0 ? kScaleOne : uint32_t(e + 127);
    return amax >= 0x7F800000u ? kScaleNaN : b;
}

// 2^-e for a scale byte of fp8_scale_byte (e <= 120, so it is a normal
// number); 0 for the NaN scale, whose values do not matter.
__device__ __forceinline__ float fp8_inverse(uint32_t byte) {
    return byte == kScaleNaN ? 0.f : __uint_as_float((254u - byte) << 23);
}

// four values, already divided by their scale (|v| <= 448), to e4m3 bytes
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d) {
    int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
    return uint32_t(__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true));
}

// The wave's scale word from the bytes of its four 16-lane groups (uniform).
__device__ __forceinline__ uint32_t fp8_scale_word(uint32_t byte) {
    return uint32_t(__builtin_amdgcn_readlane(int(byte), 0)) |
           (uint32_t(__builtin_amdgcn_readlane(int(byte), 16)) << 8) |
           (uint32_t(__builtin_amdgcn_readlane(int(byte), 32)) << 16) |
           (uint32_t(__builtin_amdgcn_readlane(int(byte), 48)) << 24);
}

// ---- launchers --------------------------------------------------------------
lynx_status launch_quantize_fp8(const uint16_t* X, int M, int K, uint8_t* q, uint8_t* scale,
                                hipStream_t stream);
lynx_status launch_quantize_fp8_weight(const uint16_t* W, int N, int K, uint8_t* q,
                                       uint8_t* scale, hipStream_t stream);
lynx_status launch_gemm_fp8(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                            const uint8_t* Ws, uint16_t* Y, int M, int N, int K,
                            hipStream_t stream);
lynx_status launch_gemm_fp8_split(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                                  const uint8_t* Ws, uint16_t* Y, int M, int N, int K,
                                  hipStream_t stream);
lynx_status launch_block_norm(const lynx_norm& d, hipStream_t stream);

}  // namespace lynx
