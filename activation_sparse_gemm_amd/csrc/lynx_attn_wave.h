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
// The kernels are made for DP = 64, 96 and 128 channels (head_dim rounded up; the rest is zero).  K and
// V tiles have rows of 64 or 128 channels (96 take 25% fewer products than 128), in 16-byte
// chunks that are permuted within the row so that neither read has bank conflicts.
#pragma once

#include <type_traits>

#include "lynx_attn.h"

namespace lynx {

// bytes of a row in LDS
template <int DP>
constexpr int kRow = DP <= 64 ? 128 : 256;
// keys to a tile: 16 KB of K, and of V
template <int DP>
constexpr int kKeys = 16384 / kRow<DP>;

// where chunk c of row r lies in its row
template <int DP>
__device__ __forceinline__ int swz_k(int r) {
    return kRow<DP> == 256 ? (r & 15) : ((r >> 1) & 7);
}
template <int DP>
__device__ __forceinline__ int swz_v(int r) {
    return kRow<DP> == 256 ? ((r & 3) << 2 | ((r >> 2) & 3)) : (((r >> 1) & 1) << 2 | ((r >> 2) & 3));
}

// The keys that an item works on, in tiles of BN: first those of the prefix (tp tiles), then the
// sequence's own.  Tiles j0 .. j0 + n - 1 are the item's.
template <int BMR, int BN>
struct AttnSpan {
    int tp, j0, n;
    __device__ __forceinline__ AttnSpan(const AttnArgs& A, const AttnItem& w) {
        const AttnPlan<BMR, BN> plan(A, w.lq, w.lk);
        const int per = sgpr(plan.per);
        // up to the last own key that the last query of the row tile sees
        const int last = min(w.lq - 1, sgpr(row_token(A, w.tile * BMR + BMR - 1)));
        const int own = A.causal ? clampi(last + w.lk - w.lq + 1, 0, w.lk) : w.lk;
        tp = (A.prefix + BN - 1) / BN;
        j0 = w.chunk * per;
        n = max(0, min(j0 + per, tp + (own + BN - 1) / BN) - j0);
    }
    // the first key of tile j within its segment, and the first row that is not there
    __device__ __forceinline__ int key(int j) const { return (j < tp ? j : j - tp) * BN; }
};

// The tiles of K, or of V, of a workgroup (or of one wave of it), one after the other, into a ring
// in LDS.  A tile is R rows, `span` rows from the one before; NW waves stage it together, 1 KB
// pieces in turn.  Rows past the item's last tile, and channels from head_dim on, become zero.
template <int DP, int R, int NW, int RING, bool IS_V>
struct TileStream {
    static constexpr int CH = kRow<DP> / 16, BYTES = R * kRow<DP>, PER = BYTES / 1024 / NW;
    static_assert(PER * NW * 1024 == BYTES, "");
    uint32_t voff[PER];
    const uint16_t *p, *own;  // the next tile; the sequence's first
    int64_t own_stride;       // elements from row to row
    uint32_t stride;          // bytes, of the present segment
    int span;
    int rows, own_rows;       // from the next tile's first row to the segment's end
    int left;                 // tiles of the prefix that are still to come
    uint32_t lds, slot;
    i32x4 rs;
    uint32_t to;

    __device__ __forceinline__ void offsets(int64_t row_stride, int D, int wave, int lane) {
        stride = uint32_t(row_stride) * 2u;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const int at = (wave * PER + i) * 64 + lane, row = at / CH;
            const int c = (at % CH) ^ (IS_V ? swz_v<DP>(row) : swz_k<DP>(row));
            voff[i] = 8 * c < D ? uint32_t(row) * stride + 16u * uint32_t(c) : 0x80000000u;
        }
    }
    // base, t: the sequence's keys of this head and their stride; pbase, pt: the prefix'.  first:
    // the stream's first row within a tile of BN rows.
    template <int BMR, int BN>
    __device__ __forceinline__ void open(const AttnSpan<BMR, BN>& span_, int prefix, int lk, const uint16_t* base,
                                         int64_t t, const uint16_t* pbase, int64_t pt, int first, int D,
                                         uint32_t lds_, int wave, int lane) {
        const int end = span_.j0 + span_.n, tp = span_.tp, j0 = span_.j0;
        span = BN;
        lds = lds_ + uint32_t(wave * PER) * 1024u;
        slot = 0;
        own = base + first * t;
        own_rows = min(lk, max(end - tp, 0) * BN) - first;
        own_stride = t;
        if (j0 < tp) {
            p = pbase + (int64_t(j0) * BN + first) * pt;
            rows = min(prefix, end * BN) - j0 * BN - first;
            left = tp - j0;
            offsets(pt, D, wave, lane);
        } else {
            p = own + int64_t(j0 - tp) * BN * t;
            rows = own_rows - (j0 - tp) * BN;
            left = -1;
            offsets(t, D, wave, lane);
        }
    }
    // The next tile's loads: begin, then each of PER pieces.
    __device__ __forceinline__ void begin(int D, int wave, int lane) {
        if (left == 0) {
            p = own;
            rows = own_rows;
            offsets(own_stride, D, wave, lane);
        }
        --left;
        const int n = min(rows, R);
        rs = make_rsrc(p, n > 0 ? uint32_t(n - 1) * stride + 2u * uint32_t(D) : 0u);
        rs = i32x4{sgpr(rs[0]), sgpr(rs[1]), sgpr(rs[2]), rs[3]};
        to = lds + slot;
        p += (int64_t(stride) * span) >> 1;
        rows -= span;
        slot = slot == (RING - 1) * BYTES ? 0 : slot + BYTES;
    }
    __device__ __forceinline__ void piece(int i) const {
        dma16(uint32_t(sgpr(int(to + uint32_t(i) * 1024u))), voff[i], rs, 0);
    }
    __device__ __forceinline__ void issue(int D, int wave, int lane) {
        begin(D, wave, lane);
#pragma unroll
        for (int i = 0; i < PER; ++i) piece(i);
    }
};

template <int DP, bool LSE>
struct AttnWave {
    static constexpr int KS = DP / 16, DB = DP / 32;
    bf16x8 q[KS];
    f32x16 o[DB];
    // m: a whole power of two, -inf before the first key that is seen; l: the sum of the
    // weights as the product with V takes them, rounded to bf16, so that a row on which one key
    // dominates is not off by that key's rounding; exact - lost: of the weights before it, for lse
    float m, l, exact, lost;
    int lane, h;

    // p: the lane's query row, or NULL
    __device__ __forceinline__ void init(const uint16_t* p, int D) {
        lane = threadIdx.x & 63;
        h = lane >> 5;
        clear();
        read_q(q, p, D);
    }
    __device__ __forceinline__ void clear() {
        m = -INFINITY;
        l = exact = lost = 0.f;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[d][e] = 0.f;
    }
    __device__ __forceinline__ void read_q(bf16x8 (&to)[KS], const uint16_t* p, int D) const {
#pragma unroll
        for (int s = 0; s < KS; ++s) {
            const int d = 16 * s + 8 * h;
            u32x4 v = {};
            if (p && d < D) v = *reinterpret_cast<const u32x4*>(p + d);
            to[s] = __builtin_bit_cast(bf16x8, v);
        }
    }

    // Where this lane's operands lie in a tile: of 32 rows of K at channels 16 i .., and of 16
    // rows of V, u = 0, 1 its rows 0-3 and 8-11 (h = 1: 4-7 and 12-15), at channels 32 db ..  The
    // permutations are exclusive ors, so the others follow from the first by one instruction.
    __device__ __forceinline__ uint32_t k_first() const {
        const int r = lane & 31;
        return uint32_t(r) * kRow<DP> + uint32_t((h ^ swz_k<DP>(r)) * 16);
    }
    __device__ __forceinline__ static uint32_t k_at(uint32_t first, int i) { return first ^ uint32_t(32 * i); }
    __device__ __forceinline__ uint32_t v_first() const {
        const int i = lane & 15, r = 4 * h + (i >> 2), c = 2 * ((lane >> 4) & 1) + ((i & 3) >> 1);
        return uint32_t(r) * kRow<DP> + uint32_t((c ^ swz_v<DP>(r)) * 16 + 8 * (i & 1));
    }
    __device__ __forceinline__ static uint32_t v_at(uint32_t first, int u, int db) {
        return (first ^ uint32_t(64 * db + 32 * u)) + uint32_t(u * 8 * kRow<DP>);
    }
    __device__ __forceinline__ static bf16x8 v_pair(const char* a, const char* b) {
        const bf16x4 x = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) bf16x4*)a);
        const bf16x4 y = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((__attribute__((address_space(3))) bf16x4*)b);
        return __builtin_shufflevector(x, y, 0, 1, 2, 3, 4, 5, 6, 7);
    }

    // Hides keys: those of this lane's query from `seen` on; key0: the block's first key
    __device__ __forceinline__ void mask(f32x16& s, int key0, int seen) const {
        const int left = seen - key0 - 4 * h;
#pragma unroll
        for (int e = 0; e < 16; ++e)
            if (8 * (e / 4) + e % 4 >= left) s[e] = -INFINITY;
    }

    // a row's maximum, or sum, from the two lanes that hold its halves
    __device__ __forceinline__ static float both_max(float v) {
        const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        return __builtin_elementwise_maximum(__uint_as_float(w[0]), __uint_as_float(w[1]));
    }
    __device__ __forceinline__ static float both_sum(float v) {
        const auto w = __builtin_amdgcn_permlane32_swap(__float_as_uint(v), __float_as_uint(v), false, false);
        return __uint_as_float(w[0]) + __uint_as_float(w[1]);
    }

    // The maximum of a row's scores, times c, in both of its lanes.  (elementwise_maximum keeps a
    // NaN: its weight is NaN whatever m is, and so is the row.)  Four chains: a chain's step
    // takes 8 cycles, others 5 (with the matrix unit at work).
    template <int NB>
    __device__ __forceinline__ static float maximum(const f32x16 (&s)[NB], float c) {
        float top[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            top[i] = s[0][i];
#pragma unroll
            for (int e = i + 4; e < 16 * NB; e += 4)
                top[i] = __builtin_elementwise_maximum(top[i], s[e / 16][e % 16]);
        }
        const float x = __builtin_elementwise_maximum(top[0], top[1]);
        return both_max(__builtin_elementwise_maximum(__builtin_elementwise_maximum(x, top[2]), top[3])) * c;
    }

    // p = 2^(c s - m).  m is raised to the whole number above a row's maximum, and what was summed
    // before scaled down, where the maximum is 2^8 above it: then l and o stay in range, and m, a
    // whole number, changes no bits of the sums' fractions.
    __device__ __forceinline__ void raise(float top) {
        const bool up = top > m + 8.f;
        if (!__ballot(up)) return;
        const float to = up ? ceilf(top) : m;
        const float f = up ? __builtin_amdgcn_exp2f(m - to) : 1.f;
        m = to;
        l *= f;
        exact *= f;
        lost *= f;
#pragma unroll
        for (int d = 0; d < DB; ++d)
#pragma unroll
            for (int e = 0; e < 16; ++e) o[d][e] *= f;
    }
    // Lanes whose row's |m| is 2^29 or more after raise(top).  (Where m is -2^29 or below and top is not,
    // m is raised: m + 8 is m there.  From 2^24 on m + 8 may still be more, and top between the two.)
    static constexpr float kFar = 536870912.f;
    __device__ __forceinline__ uint64_t far(float top) const { return __ballot(fmaxf(fabsf(top), m) >= kFar); }
    __device__ __forceinline__ bool near() const { return fabsf(m) < kFar; }
    __device__ __forceinline__ static float apart(float v, float c, float from) {
#pragma clang fp contract(off)
        const float t = v * c;
        return t - from;
    }

    // A tile's sums of weights, in four parts, since a chain's step takes longer.
    struct Sums {
        float rounded[4] = {0.f, 0.f, 0.f, 0.f}, exact[4] = {0.f, 0.f, 0.f, 0.f};
    };
    // Scores of 32 keys to weights, P^T's operand for two steps of 16 keys, and their sums
    __device__ __forceinline__ void weights(f32x16& s, float c, u32x4 (&p)[2], Sums& sum) {
        typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
        const bf16x2 one = {static_cast<__bf16>(1.f), static_cast<__bf16>(1.f)};
        const float base = near() ? m : 0.f;
#pragma unroll
        for (int e = 0; e < 16; ++e) s[e] = __builtin_amdgcn_exp2f(fmaf(s[e], c, -base));
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t w = pack_bf16(s[2 * i], s[2 * i + 1]);
            sum.rounded[i % 4] =
                __builtin_amdgcn_fdot2_f32_bf16(__builtin_bit_cast(bf16x2, w), one, sum.rounded[i % 4], false);
            if constexpr (LSE) sum.exact[i % 4] += s[2 * i] + s[2 * i + 1];
            p[i / 4][i % 4] = w;
        }
    }
    // A tile's sums to the row's: once a tile, since weights that are alike all round the same way in a
    // sum that has grown.  lse's sum keeps what such an addition loses (Kahan), so that its error does
    // not grow with the keys: lse of 262144 equal scores was 2e-3 off with every weight added singly, and is
    // 2e-6 off so.  (l goes with o, which the matrix instructions sum in fp32, 16 keys at a time.)
    __device__ __forceinline__ void add(const Sums& t) {
        l += (t.rounded[0] + t.rounded[1]) + (t.rounded[2] + t.rounded[3]);
        if constexpr (LSE) {
            const float y = ((t.exact[0] + t.exact[1]) + (t.exact[2] + t.exact[3])) - lost, n = exact + y;
            lost = (n - exact) - y;
            exact = n;
        }
    }
};

// The products of a wave's 32 rows with tiles of BN keys in LDS: S^T = K Q^T of one tile together
// with O^T += V^T P^T of the tile before, which leaves neither waiting for itself.  Operands are
// read AHEAD products early.  k, v: LDS offsets of a tile plus the lane's k_first or v_first.
template <int DP, int BN, bool LSE>
struct AttnTile : AttnWave<DP, LSE> {
    using W = AttnWave<DP, LSE>;
    static constexpr int NB = BN / 32, NM = NB * W::KS, AHEAD = 4;
    static_assert(NM == 2 * NB * W::DB, "as many products of either kind");
    f32x16 s[NB];
    u32x4 p[NB][2];
    bf16x8 kf[NM], vf[NM];

    __device__ __forceinline__ void read(const char* smem, uint32_t k, uint32_t v, int i, bool qk, bool pv) {
        if (qk)
            kf[i] = *reinterpret_cast<const bf16x8*>(smem + W::k_at(k, i / NB) + (i % NB) * (32 * kRow<DP>));
        if (pv) {
            const char* at = smem + (i / W::DB) * (16 * kRow<DP>);
            vf[i] = W::v_pair(at + W::v_at(v, 0, i % W::DB), at + W::v_at(v, 1, i % W::DB));
        }
    }
    template <bool QK, bool PV>
    __device__ __forceinline__ void ahead(const char* smem, uint32_t k, uint32_t v) {
#pragma unroll
        for (int i = 0; i < AHEAD; ++i) read(smem, k, v, i, QK, PV);
    }
    // between(i) is called before products i, i = 0 .. NM - 1
    template <bool QK, bool PV, class Between>
    __device__ __forceinline__ void multiply(const char* smem, uint32_t k, uint32_t v, Between between) {
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            between(i);
            if (i + AHEAD < NM) read(smem, k, v, i + AHEAD, QK, PV);
            if constexpr (QK) {
                f32x16 c = s[i % NB];
                if (i < NB) {
#pragma unroll
                    for (int e = 0; e < 16; ++e) c[e] = 0.f;
                }
                s[i % NB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(kf[i], W::q[i / NB], c, 0, 0, 0);
            }
            if constexpr (PV) {
                const int t = i / W::DB, d = i % W::DB;
                W::o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(vf[i], __builtin_bit_cast(bf16x8, p[t / 2][t % 2]),
                                                                 W::o[d], 0, 0, 0);
            }
        }
        constexpr int reads = (QK ? 1 : 0) + (PV ? 2 : 0), products = (QK ? 1 : 0) + (PV ? 1 : 0);
#pragma unroll
        for (int i = 0; i < NM; ++i) {
            if (i + AHEAD < NM) __builtin_amdgcn_sched_group_barrier(0x100, reads, 0);
            __builtin_amdgcn_sched_group_barrier(0x008, products, 0);
        }
    }
    template <bool QK, bool PV>
    __device__ __forceinline__ void multiply(const char* smem, uint32_t k, uint32_t v) {
        multiply<QK, PV>(smem, k, v, [](int) {});
    }

    // The halves of a word of two bf16 that are no finite numbers
    __device__ __forceinline__ static uint32_t odd_halves(uint32_t w) {
        return ((w & 0x7F80u) == 0x7F80u ? 0xFFFFu : 0u) | ((w & 0x7F800000u) == 0x7F800000u ? 0xFFFF0000u : 0u);
    }
    // O^T += V^T P^T where rows do not see every key (left: how many of the tile's a lane's row
    // does).  A hidden key's weight is 0, but its value may be infinite or NaN, and 0 times
    // that is NaN: such values are taken as 0, and added, key by key, to the rows that see them.
    __device__ __forceinline__ void multiply_hidden(const char* smem, uint32_t v, int left) {
        typedef unsigned short u16x2 __attribute__((ext_vector_type(2)));
        auto step = [&](int t, u32x4 (&w)[W::DB]) {
            const char* at = smem + t * (16 * kRow<DP>);
#pragma unroll
            for (int d = 0; d < W::DB; ++d)
                w[d] = __builtin_bit_cast(u32x4, W::v_pair(at + W::v_at(v, 0, d), at + W::v_at(v, 1, d)));
        };
        u32x4 next[W::DB];
        step(0, next);
#pragma unroll
        for (int t = 0; t < 2 * NB; ++t) {
            u16x2 top = {0, 0};
            u32x4 w[W::DB];
            const u32x4 pw = p[t / 2][t % 2];
#pragma unroll
            for (int d = 0; d < W::DB; ++d) w[d] = next[d];
            if (t + 1 < 2 * NB) step(t + 1, next);
#pragma unroll
            for (int d = 0; d < W::DB; ++d)
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, w[d][e] & 0x7F807F80u));
            if (__ballot(top[0] == 0x7F80 || top[1] == 0x7F80)) {
#pragma unroll
                for (int d = 0; d < W::DB; ++d) {
                    add_odd(w[d], pw, d, left - 16 * t);
#pragma unroll
                    for (int e = 0; e < 4; ++e) w[d][e] &= ~odd_halves(w[d][e]);
                }
            }
#pragma unroll
            for (int d = 0; d < W::DB; ++d)
                W::o[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, w[d]),
                                                                 __builtin_bit_cast(bf16x8, pw), W::o[d], 0, 0, 0);
        }
    }
    // The values among w (16 keys, channels 32 d ..) that are no finite numbers, times the weights
    // pw, to the rows that see them: those with more than the key's number `left`
    __device__ __forceinline__ void add_odd(const u32x4& w, const u32x4& pw, int d, int left) {
        for (int k = 0; k < 16; ++k) {  // slot k % 8 of half k / 8
            u32x4 a, b;
#pragma unroll
            for (int e = 0; e < 4; ++e) {
                const uint32_t half = k & 1 ? 0xFFFF0000u : 0xFFFFu;
                const uint32_t keep = W::h == k >> 3 && e == (k & 7) >> 1 ? half : 0u;
                a[e] = w[e] & keep & odd_halves(w[e]);
                b[e] = pw[e] & keep;
            }
            f32x16 c;
#pragma unroll
            for (int e = 0; e < 16; ++e) c[e] = 0.f;
            c = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a),
                                                       __builtin_bit_cast(bf16x8, b), c, 0, 0, 0);
            const bool sees = 4 * (k >> 3) + (k & 3) + 8 * ((k & 7) >> 2) < left;
#pragma unroll
            for (int e = 0; e < 16; ++e) W::o[d][e] += sees ? c[e] : 0.f;
        }
    }
    // Raises m to a tile's scores, before their weights.  A multiply-add takes c s as it is, and m is
    // fp32: from 2^24 on, c s - m of a row's largest score is what m has lost, up to half its last
    // place.  That is 2^4 below 2^29, which changes all weights of a row alike, but past 2^7 from 2^31
    // on (weights of infinity, or of 0 alone).  In rows past 2^29 c s is rounded as m was, and the
    // scores become those that are as far from 0 as c s was from m.
    __device__ __forceinline__ void relate(float top, float c) {
        // (early, since a branch waits for its condition: 16384 x 16384 x 8 heads 980 us without, 993 so,
        // 998 with the condition after m is raised)
        const uint64_t rows = W::far(top);
        W::raise(top);
        if (rows == 0) return;
        const bool mine = !W::near() && W::m != -INFINITY;
        const float back = 1.f / c;
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
            for (int e = 0; e < 16; ++e) s[b][e] = mine ? W::apart(s[b][e], c, W::m) * back : s[b][e];
    }
    // Hides keys from `seen` on; key0: the tile's first
    __device__ __forceinline__ void hide(int key0, int seen) {
#pragma unroll
        for (int b = 0; b < NB; ++b) W::mask(s[b], key0 + 32 * b, seen);
    }
};

// The query row's place: token and head of row `row` of an item, or false where there is none.
__device__ __forceinline__ bool attn_row(const AttnArgs& A, const AttnItem& w, int row, int& token,
                                         int& head) {
    const int t = row_token(A, row);
    token = w.q0 + t;
    head = w.kvh * A.group + (row - t * A.group);
    return t < w.lq;
}
__device__ __forceinline__ int64_t attn_q_offset(const AttnArgs& A, int token, int head) {
    if (A.addr_len == 0) return token * A.q_t + head * A.q_h;
    const int b = token / A.addr_len;
    return b * A.q_b + (token - b * A.addr_len) * A.q_t + head * A.q_h;
}
__device__ __forceinline__ int64_t attn_o_offset(const AttnArgs& A, int token, int head) {
    if (A.addr_len == 0) return token * A.o_t + head * A.o_h;
    const int b = token / A.addr_len;
    return b * A.o_b + (token - b * A.addr_len) * A.o_t + head * A.o_h;
}

// Writes a wave's rows (row0 ..): to out and lse, or as a chunk's partial result.
template <int DP, bool LSE>
__device__ __forceinline__ void store_rows(const AttnArgs& A, const AttnItem& w, const AttnWave<DP, LSE>& W,
                                           int row0, bool part) {
    const float l = W.both_sum(W.l), le = LSE ? W.both_sum(W.exact) : 0.f;
    int token, head;
    if (!attn_row(A, w, row0 + (W.lane & 31), token, head)) return;
    const int64_t row = int64_t(token) * A.heads + head;
    if (part) {
        const int64_t slot = row * A.slots + A.slot0 + w.chunk;
        float* o = A.part_o + slot * A.D;
#pragma unroll
        for (int d = 0; d < DP / 32; ++d)
#pragma unroll
            for (int g = 0; g < 4; ++g) {
                const int at = 32 * d + 8 * g + 4 * W.h;
                if (at < A.D)
                    *reinterpret_cast<f32x4*>(o + at) =
                        f32x4{W.o[d][4 * g], W.o[d][4 * g + 1], W.o[d][4 * g + 2], W.o[d][4 * g + 3]};
            }
        if (W.h == 0) {
            A.part_ml[slot] = float4{W.m, l, le, 0.f};
            if (w.chunk == 0 && A.part_n) A.part_n[row] = w.chunks;
        }
        return;
    }
    // A lane holds channels 8 g + 4 h .. + 3 of its row: of two groups g, it keeps one and gets its
    // other half from the row's other lane, 16 bytes to a store
    const float inv = l == 0.f ? 0.f : 1.f / l;
    uint16_t* o = A.out + attn_o_offset(A, token, head);
#pragma unroll
    for (int d = 0; d < DP / 32; ++d)
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
            uint32_t w[2][2];
#pragma unroll
            for (int i = 0; i < 2; ++i)
#pragma unroll
                for (int e = 0; e < 2; ++e)
                    w[i][e] = pack_bf16(W.o[d][4 * (g + i) + 2 * e] * inv, W.o[d][4 * (g + i) + 2 * e + 1] * inv);
            const auto lo = __builtin_amdgcn_permlane32_swap(w[0][0], w[1][0], false, false);
            const auto hi = __builtin_amdgcn_permlane32_swap(w[0][1], w[1][1], false, false);
            const int at = 32 * d + 8 * (g + W.h);
            if (at < A.D) *reinterpret_cast<u32x4*>(o + at) = u32x4{lo[0], hi[0], lo[1], hi[1]};
        }
    if (W.h == 0) {
        if constexpr (LSE) A.lse[row] = le == 0.f ? -INFINITY : (W.m + log2f(le)) * kLn2;
        if (A.slots > 0 && w.chunk == 0) A.part_n[row] = 1;
    }
}

// K's (V's) streams of an item
template <class S, int BMR, int BN>
__device__ __forceinline__ void open_stream(S& s, const AttnArgs& A, const AttnItem& w, const AttnSpan<BMR, BN>& span,
                                            bool v, int first, uint32_t lds, int wave, int lane) {
    const int64_t t = v ? A.v_t : A.k_t, pt = v ? A.pv_t : A.pk_t;
    const uint16_t* base = (v ? A.v : A.k) + (A.cu_k ? w.k0 * t : w.seq * (v ? A.v_b : A.k_b)) +
                           w.kvh * (v ? A.v_h : A.k_h);
    const uint16_t* pbase = (v ? A.pv : A.pk) + w.kvh * (v ? A.pv_h : A.pk_h);
    s.open(span, A.prefix, w.lk, base, t, pbase, pt, first, A.D, lds, wave, lane);
}

// What a wave's rows see of the sequence's own lk keys: a lane's row `seen`, all of them `all`, any
// of them `any`.  none: the wave has no row.
struct AttnView {
    int seen, all, any, lk;
    bool none;
    __device__ __forceinline__ AttnView(const AttnArgs& A, const AttnItem& w, int row0, int lane) {
        auto keys = [&](int t) { return A.causal ? clampi(t + w.lk - w.lq + 1, 0, w.lk) : w.lk; };
        const int t0 = sgpr(row_token(A, row0)), t1 = min(w.lq - 1, sgpr(row_token(A, row0 + 31)));
        seen = keys(row_token(A, row0 + (lane & 31)));
        all = keys(t0);
        any = keys(t1);
        lk = w.lk;
        none = t0 >= w.lq;
    }
    // of these, the first ones of which all rows see every key.  (Not: of which they see the same keys.
    // 32 rows of one token do, and their last tile still holds the keys of later tokens.)
    template <int BMR, int BN>
    __device__ __forceinline__ int plain(const AttnSpan<BMR, BN>& span) const {
        return all < lk ? clampi(span.tp + all / BN - span.j0, 0, span.n) : span.n;
    }
    // the item's tiles that the wave works on: the first ones
    template <int BMR, int BN>
    __device__ __forceinline__ int tiles(const AttnSpan<BMR, BN>& span) const {
        return none ? 0 : clampi(span.tp + (any + BN - 1) / BN - span.j0, 0, span.n);
    }
};

// Calls go(channels, lse, causal) with the constants of the kernel that `a` needs.
template <class Go>
void attn_variant(const AttnArgs& a, Go go) {
    using yes = std::integral_constant<bool, true>;
    using no = std::integral_constant<bool, false>;
    auto with = [&](auto dp) {
        if (a.lse) a.causal ? go(dp, yes{}, yes{}) : go(dp, yes{}, no{});
        else a.causal ? go(dp, no{}, yes{}) : go(dp, no{}, no{});
    };
    if (a.D <= 64) with(std::integral_constant<int, 64>{});
    else if (a.D <= 96) with(std::integral_constant<int, 96>{});
    else with(std::integral_constant<int, 128>{});
}

}  // namespace lynx
