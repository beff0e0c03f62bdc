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

// 16-byte chunk swizzle of 128-byte LDS rows that 16 x 16 x 128 fragments are read from
// (lane l: row l % 16, chunk l / 16 or 4 + l / 16).  A 16-byte read is served in groups
// of 16 lanes that hold rows 0-3 and 12-15 of one chunk and 4-11 of the next (or the
// other way round), not in order: rows of a parity (half the banks each) then fall on
// eight unlike chunks.  A row & 7 swizzle had 2-way conflicts on every read.
__device__ __forceinline__ int fp8_swz(int row) { return (row >> 1) & 7; }

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

// The fp32 number that the conversions below divide by for a scale byte: they use
// its exponent field alone.  (255, the NaN scale, gives values that do not matter.)
__device__ __forceinline__ float fp8_divisor(uint32_t byte) { return __uint_as_float(byte << 23); }

// four values to e4m3 bytes, divided by 2^e (exactly) and rounded to nearest even
__device__ __forceinline__ uint32_t fp8_pack4(float a, float b, float c, float d, float divisor) {
    typedef short i16x2 __attribute__((ext_vector_type(2)));
    i16x2 w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, a, b, divisor, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, c, d, divisor, true);
    return __builtin_bit_cast(uint32_t, w);
}
// the same from two words of bf16 pairs
__device__ __forceinline__ uint32_t fp8_pack4(uint32_t ab, uint32_t cd, float divisor) {
    typedef short i16x2 __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    i16x2 w = {0, 0};
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2, ab), divisor, false);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(bf16x2, cd), divisor, true);
    return __builtin_bit_cast(uint32_t, w);
}

// fp32 bits of the largest magnitude of eight bf16
__device__ __forceinline__ uint32_t fp8_amax8(const u32x4& v) {
    typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
    u16x2 m = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, v[i] & 0x7FFF7FFFu));
    return uint32_t(m[0] > m[1] ? m[0] : m[1]) << 16;
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

// Product kernels (launch_gemm_fp8 chooses).  _few: M <= kFewRows; _mid: few output
// tiles; each from the 8-bit operand, or from bf16 X quantised on the way in.
constexpr int kFewRows = 16;
constexpr int kFewQuant = 32768;  // elements of X that _few quantises

// _few, unless there are enough columns to fill the chip with larger tiles, which read
// X less often: 16 x 3072 -> 3072 5.1 us, in 32 x 32 tiles 6.4; -> 9216 10.8, in 32 x 64
// tiles 7.9; 4 rows -> 9216 8.4.
inline bool fp8_is_few(int64_t M, int64_t N) { return M <= 8 || (M <= kFewRows && N < 8192); }

inline int64_t fp8_tiles(int64_t M, int64_t N, int64_t tm, int64_t tn) {
    return (M + tm - 1) / tm * ((N + tn - 1) / tn);
}

// Whether lynx_linear_fp8 quantises inside the product, in the same order of sums as the
// product has on a 256-unit device (so that its results are those of quantiser and
// product).  It costs a product 1.4 us per 1024 of K in 32 x 32 tiles, 2.1 in 32 x 64 ones
// and 3.6 with two of them to a unit, and saves 0.55 us per million elements of X, which
// is then read once, and a kernel: 2.2 us, and 3 us of the host (5 with the workspace,
// from Python), which bound short calls unless they are replayed from a graph.  1.3 us
// are counted for that.  In one kernel and apart, us: from a graph 64 x 1024 -> 1024 5.6
// and 6.4, 64 x 2048 -> 2048 8.3 and 7.4 (called one by one 7.9 and 11.6), 128 x 1472 ->
// 3072 7.9 and 7.8 (7.4 and 11.6), 768 x 1024 -> 1024 8.8 and 7.9, 9216 x 640 -> 64 7.2 and
// 10.4; 4096 x 3072 -> 64 11.0 and 15.0.
enum class Fp8Fuse { no, few, mid32, mid64 };
inline Fp8Fuse fp8_fuse(int64_t M, int64_t N, int64_t K) {
    if (fp8_is_few(M, N)) return M * K <= kFewQuant ? Fp8Fuse::few : Fp8Fuse::no;
    const int64_t apart = 3500000 + M * K * 11 / 20;  // picoseconds
    if (fp8_tiles(M, N, 32, 32) <= 256) return K * 1400 < apart ? Fp8Fuse::mid32 : Fp8Fuse::no;
    const int64_t tiles = fp8_tiles(M, N, 32, 64);
    if (tiles <= 512 && K * (tiles <= 256 ? 2050 : 3600) < apart) return Fp8Fuse::mid64;
    return Fp8Fuse::no;
}

lynx_status launch_gemm_fp8_few(const void* X, const uint8_t* Xs, const uint8_t* Wq,
                                const uint8_t* Ws, uint16_t* Y, int M, int N, int K,
                                hipStream_t stream);
lynx_status launch_gemm_fp8_mid_quant(const uint16_t* X, const uint8_t* Wq, const uint8_t* Ws,
                                      uint16_t* Y, int M, int N, int K, Fp8Fuse how,
                                      hipStream_t stream);
// Takes the problem if its tile counts suit it; *taken says whether it did.
lynx_status launch_gemm_fp8_mid(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                                const uint8_t* Ws, uint16_t* Y, int M, int N, int K, int cus,
                                bool* taken, hipStream_t stream);
lynx_status launch_block_norm(const lynx_norm& d, hipStream_t stream);

}  // namespace lynx
