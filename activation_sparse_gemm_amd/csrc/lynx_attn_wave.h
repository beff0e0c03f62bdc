// One wave's part of the attention kernels: 32 QB query rows against a tile of keys in LDS.
//
// The products are transposed: S^T = K Q^T, then O^T += V^T P^T, both on
// v_mfma_f32_32x32x16_bf16, whose result has a query in each lane (lane & 31) and keys, or
// channels of O, in its registers.  So a row's maximum, sum and factor are a lane's own
// (two lanes', h = lane / 32, which hold half the keys each), and S^T's registers, rounded to
// bf16, are P^T's operand as they stand: registers 8 t .. 8 t + 7 of a 32-key block hold
// keys 16 t + {4 h .. 4 h + 3, 8 + 4 h .. 8 + 4 h + 3}, and the order of keys inside a product
// is free as long as V^T's operand has the same one.  V lies in LDS by rows of keys;
// ds_read_b64_tr_b16 transposes it on the way: of 16 lanes, lane i supplies the address of
// channels 4 (i % 4) .. + 3 of key i / 4, and receives channel i of the four keys.
//
// K and V tiles have rows of DP channels (head_dim rounded up; the rest is zero), in 16-byte
// chunks that are permuted within the row so that neither read has bank conflicts.
#pragma once

#include "lynx_attn.h"

namespace lynx {

// where chunk c of row r lies in its row
template <int DP>
__device__ __forceinline__ int swz_k(int r) {
    return DP == 128 ? (r & 15) : ((r >> 1) & 7);
}
template <int DP>
__device__ __forceinline__ int swz_v(int r) {
    return DP == 128 ? ((r & 3) << 2 | ((r >> 2) & 3)) : (((r >> 1) & 1) << 2 | ((r >> 2) & 3));
}

// Stages BN rows of K or V into LDS: waves W0 .. W0 + NW - 1 of the workgroup take 1 KB
// pieces in turn.  Rows from `rows` on and channels from D on become zero.
template <int DP, int BN, int NW, bool IS_V>
struct AttnStage {
    static constexpr int CH = DP / 8, PIECES = BN * DP * 2 / 1024, PER = PIECES / NW;
    static_assert(PIECES % NW == 0, "");
    uint32_t voff[PER];
    uint32_t tile_bytes;  // from one tile to the next
    uint32_t stride;      // bytes from one row to the next

    __device__ __forceinline__ void init(int64_t row_stride, int D, int wave, int lane) {
        stride = uint32_t(row_stride) * 2u;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = (wave * PER + i) * 64 + lane, row = at / CH;
            const int c = (at % CH) ^ (IS_V ? swz_v<DP>(row) : swz_k<DP>(row));
            voff[i] = 8 * c < D ? uint32_t(row) * stride + 16u * uint32_t(c) : 0x80000000u;
        }
    }
    // base: the tile's first row; rows: how many of its rows there are (others read zero)
    __device__ __forceinline__ void load(const uint16_t* base, int rows, int D, uint32_t lds,
                                         int wave) const {
        const int n = clampi(rows, 0, BN);
        i32x4 rs = make_rsrc(base, n > 0 ? uint32_t(n - 1) * stride + 2u * uint32_t(D) : 0u);
        rs = i32x4{sgpr(rs[0]), sgpr(rs[1]), sgpr(rs[2]), rs[3]};
#pragma unroll
        for (int i = 0; i < PER; ++i)
            dma16(uint32_t(sgpr(int(lds + uint32_t(wave * PER + i) * 1024u))), voff[i], rs, 0);
    }
};

template <int DP, int QB, bool LSE>
struct AttnWave {
    static constexpr int KS = DP / 16, DB = DP / 32;
    bf16x8 q[QB][KS];
    f32x16 o[QB][DB];
    // m: a whole power of two, -inf before the first key that is seen; l: the sum of the
    // weights as the product with V takes them, rounded to bf16, so that a row on which one key
    // dominates is not off by that key's rounding; exact: of the weights before it, for lse
    float m[QB], l[QB], exact[LSE ? QB : 1];
    uint32_t ka, va;     // LDS offsets of this lane's operands
    int lane, h;

    __device__ __forceinline__ void init(int lane_) {
        lane = lane_;
        h = lane >> 5;
        ka = uint32_t(lane & 31);
        va = 0;
#pragma unroll
        for (int b = 0; b < QB; ++b) {
            m[b] = -INFINITY;
            l[b] = 0.f;
            if constexpr (LSE) exact[b] = 0.f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[b][d][e] = 0.f;
        }
    }

    // this lane's query of block b; p: its row, or NULL
    __device__ __forceinline__ void load_q(int b, const uint16_t* p, int D) {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = 16 * s + 8 * h;
            u32x4 v = {};
            if (p && d < D) v = *reinterpret_cast<const u32x4*>(p + d);
            q[b][s] = __builtin_bit_cast(bf16x8, v);
        }
    }

    // S^T of the 32 keys from row `row` of the K tile at LDS byte `lds`
    __device__ __forceinline__ void scores(const char* smem, uint32_t lds, int row, f32x16 (&s)[QB]) {
#pragma unroll
        for (int b = 0; b < QB; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[b][e] = 0.f;
        const int r = lane & 31;
#pragma unroll
        for (int i = 0; i < KS; ++i) {
            const uint32_t off = uint32_t(r) * (DP * 2) + uint32_t(((2 * i + h) ^ swz_k<DP>(r)) * 16);
            const bf16x8 k =
                *reinterpret_cast<const bf16x8*>(smem + lds + uint32_t(row) * (DP * 2) + off);
#pragma unroll
            for (int b = 0; b < QB; ++b)
                s[b] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k, q[b][i], s[b], 0, 0, 0);
        }
    }

    // V^T's operand: channels 32 db .., keys row + 16 t ..
    __device__ __forceinline__ bf16x8 v_operand(const char* smem, uint32_t lds, int row, int db) {
        const int i = lane & 15, dsub = (lane >> 4) & 1;
        bf16x4 part[2];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int r = 8 * u + 4 * h + (i >> 2);
            const int c = 4 * db + 2 * dsub + ((i & 3) >> 1);
            const uint32_t off =
                uint32_t(r) * (DP * 2) + uint32_t((c ^ swz_v<DP>(r)) * 16 + 8 * (i & 1));
            part[u] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                (__attribute__((address_space(3))) bf16x4*)(smem + lds + uint32_t(row) * (DP * 2) + off));
        }
        return __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
    }

    // Hides keys: those of this lane's query from `seen` on; key0: the block's first key
    __device__ __forceinline__ void mask(f32x16& s, int key0, int seen) const {
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (key0 + 8 * (e / 4) + 4 * h + e % 4 >= seen) s[e] = -INFINITY;
    }

    // a row's maximum, or sum, from the two lanes that hold its halves
    __device__ __forceinline__ static float both_max(float v) {
        const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        return fmaxf(__uint_as_float(w[0]), __uint_as_float(w[1]));
    }
    __device__ __forceinline__ static float both_sum(float v) {
        const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        return __uint_as_float(w[0]) + __uint_as_float(w[1]);
    }

    // Scores to weights, in place, for NKB blocks of 32 keys.  p = 2^(c s - m); m is raised,
    // and what was summed before scaled down, where a row's maximum is 2^8 above it: then l and
    // o stay in range, and m, a whole number, changes no bits of the sums' fractions.
    template <int NKB>
    __device__ __forceinline__ void softmax(int b, f32x16 (&s)[NKB][QB], float c) {
        float top = s[0][b][0];
#pragma unroll
        for (int n = 0; n < NKB; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) top = fmaxf(top, s[n][b][e]);
        top = both_max(top) * c;
        const bool raise = top > m[b] + 8.f;
        if (__ballot(raise)) {
            const float to = raise ? ceilf(top) : m[b];
            const float f = raise ? __builtin_amdgcn_exp2f(m[b] - to) : 1.f;
            m[b] = to;
            l[b] *= f;
            if constexpr (LSE) exact[b] *= f;
#pragma unroll
            for (int d = 0; d < DB; ++d)
#pragma unroll
                for (int e = 0; e < 16; ++e) o[b][d][e] *= f;
        }
        const float base = m[b] == -INFINITY ? 0.f : m[b];
#pragma unroll
        for (int n = 0; n < NKB; ++n)
#pragma unroll
            for (int e = 0; e < 16; ++e) {
                s[n][b][e] = __builtin_amdgcn_exp2f(fmaf(s[n][b][e], c, -base));
                if constexpr (LSE) exact[b] += s[n][b][e];
            }
    }

    __device__ __forceinline__ static bf16x8 weights(const f32x16& s, int t, float& l) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const bf16x2 one = {static_cast<__bf16>(1.f), static_cast<__bf16>(1.f)};
        u32x4 w;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const uint32_t p = pack_bf16(s[8 * t + 2 * i], s[8 * t + 2 * i + 1]);
            l = __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, p), one, l, false);
            w[i] = p;
        }
        return __builtin_bit_cast(bf16x8, w);
    }

    // O^T += V^T P^T over the 32 keys from row `row` of the V tile
    __device__ __forceinline__ void accumulate(const char* smem, uint32_t lds, int row, const f32x16 (&s)[QB]) {
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            bf16x8 p[QB];
#pragma unroll
            for (int b = 0; b < QB; ++b) p[b] = weights(s[b], t, l[b]);
#pragma unroll
            for (int d = 0; d < DB; ++d) {
                const bf16x8 v = v_operand(smem, lds, row + 16 * t, d);
#pragma unroll
                for (int b = 0; b < QB; ++b)
                    o[b][d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(v, p[b], o[b][d], 0, 0, 0);
            }
        }
    }
};

// The query row's place: token and head of row `row` of an item, or false where there is none.
__device__ __forceinline__ bool attn_row(const AttnArgs& A, const AttnItem& w, int row, int& token,
                                         int& head) {
    const int t = row / A.group;
    token = w.q0 + t;
    head = w.kvh * A.group + (row - t * A.group);
    return t < w.lq;
}
__device__ __forceinline__ int64_t attn_q_offset(const AttnArgs& A, int token, int head) {
    const int b = token / A.addr_len;
    return b * A.q_b + (token - b * A.addr_len) * A.q_t + head * A.q_h;
}
__device__ __forceinline__ int64_t attn_o_offset(const AttnArgs& A, int token, int head) {
    const int b = token / A.addr_len;
    return b * A.o_b + (token - b * A.addr_len) * A.o_t + head * A.o_h;
}

}  // namespace lynx
