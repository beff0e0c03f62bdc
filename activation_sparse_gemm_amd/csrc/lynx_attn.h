// Internal declarations of the attention path: the kernels' arguments, the order in which
// workgroups take their work, and the launchers (validated arguments only).
#pragma once

#include "lynx_dma.h"

namespace lynx {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    typedef float f32x2_t __attribute__((ext_vector_type(2)));
    typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));
    return __builtin_bit_cast(uint32_t, __builtin_convertvector(f32x2_t{a, b}, bf16x2_t));
}

constexpr int kMaxChunks = 128;  // of a pass
constexpr int kNearTiles = 5;    // of keys, that the kernel for few keys has room for

// Arguments of an attention kernel.  Query rows of one sequence and key head are numbered
// token * group + head in group, so that the heads that share a key head share its tiles.
//
// Keys are cut into tiles (the prefix' tiles first, then the sequence's own), tiles into
// chunks of at least chunk_tiles, at most chunk_max of them to a sequence.  Work is the list
// of (sequence, key head, row tile, chunk).  Where slots > 0 a chunk's result goes to the
// partial sums: row's slot slot0 + chunk, part_n[row] chunks; attn_join_kernel adds them up.  A
// sequence of one chunk goes straight to out, unless force_part.
struct AttnArgs {
    const uint16_t *q, *k, *v, *pk, *pv;
    const int *cu_q, *cu_k;
    uint16_t* out;
    float* lse;
    float* part_o;    // [row][slot][D]
    float4* part_ml;  // [row][slot]: m in powers of two, l, l of unrounded weights (with lse)
    int* part_n;      // [row]; NULL in the pass over a prefix, whose chunks are the same for all rows
    int64_t q_b, q_t, q_h, o_b, o_t, o_h;
    int64_t k_b, k_t, k_h, v_b, v_t, v_h, pk_t, pk_h, pv_t, pv_h;
    int batch, heads, kv_heads, group, D;
    int tokens_q, tokens_k, prefix;
    int len_q, len_k;    // uniform form: tokens of a sequence
    int addr_len;        // tokens of q and out that are q_t apart; 0: all
    int slots, slot0, force_part, chunk_tiles, chunk_max;
    int classes;         // gcd(kv_heads, 8)
    int group_shift;     // log2(group), or -1
    int pieces;          // uniform form: pieces of a sequence to a key head (few keys: shares of its rows)
    float c;             // scale * log2(e)
    int causal;
};

// A workgroup's piece of work.
struct AttnItem {
    int kvh;             // key head
    int q0, lq;          // first query token, query tokens
    int64_t k0;          // first key token
    int lk;              // key tokens
    int tile, chunk, chunks;
    int seq;
};

__device__ __forceinline__ int clampi(int v, int lo, int hi) { return min(max(v, lo), hi); }

// a value that every lane holds, as a scalar
__device__ __forceinline__ int sgpr(int v) { return __builtin_amdgcn_readfirstlane(v); }

// token of a row number (a division costs 30 instructions)
__device__ __forceinline__ int row_token(const AttnArgs& A, int row) {
    return A.group_shift >= 0 ? row >> A.group_shift : row / A.group;
}

// inclusive sum over the first n lanes of a wave (those behind them hold 0: the last lane has
// the whole sum)
__device__ __forceinline__ int wave_scan(int v, int lane, int n) {
    for (int d = 1; d < min(n, 64); d *= 2) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// Row tiles and chunks of a sequence.
template <int BM, int BN>
struct AttnPlan {
    int tiles, chunks, per;  // per: key tiles of a chunk
    template <class Args>
    __host__ __device__ __forceinline__ AttnPlan(const Args& A, int lq, int lk) {
        tiles = (lq * A.group + BM - 1) / BM;
        const int kt = (A.prefix + BN - 1) / BN + (lk + BN - 1) / BN;
        if (A.chunk_max == 1) {
            per = kt > 1 ? kt : 1;
            chunks = 1;
        } else {
            per = (kt + A.chunk_max - 1) / A.chunk_max;
            // (few rows: longer chunks where a sequence has several row tiles after all, so that
            // these do not add to the length of the work list)
            const int64_t least = int64_t(A.chunk_tiles) * (BM == 32 ? tiles : 1);
            if (per < least) per = least < kt ? int(least) : kt;
            chunks = kt > 0 ? (kt + per - 1) / per : 1;
        }
    }
};

// The piece of work of workgroup `block`; false if there is none.  Uniform over the workgroup.
// Workgroups of one XCD (their number mod 8) take the same key heads, one after the other, so that
// its L2 holds the keys and values that its workgroups read; where there are fewer key heads than
// XCDs several share a head.  Within a head sequences follow one another, those of most keys first
// where there are up to 64 (12 of 32 .. 4096 causal tokens, 32/8 x 128: 135 -> 130 us; not for few
// rows, whose pieces are of one size), and a sequence's row tiles come last tile first: under a
// causal mask these have the most keys, and the light ones fill the end.
template <int BM, int BN>
__device__ __forceinline__ bool attn_item(const AttnArgs& A, int block, AttnItem& w) {
    const int lane = threadIdx.x & 63;
    // of sequence s: its range of tokens, and how many pieces it has to a key head
    struct Range {
        int q0, lq, k0, lk;
    };
    auto range = [&](int s) {
        Range r;
        r.q0 = clampi(A.cu_q[s], 0, A.tokens_q);
        r.lq = clampi(A.cu_q[s + 1], r.q0, A.tokens_q) - r.q0;
        r.k0 = clampi(A.cu_k[s], 0, A.tokens_k);
        r.lk = clampi(A.cu_k[s + 1], r.k0, A.tokens_k) - r.k0;
        return r;
    };
    // (A grid has fewer workgroups than `most`.  Offsets that go back and forth make sequences of the
    // same tokens, of which 65536 have more pieces in all than an int holds; these are cut off, and so
    // are sums below, which then stay below 2^31.)
    constexpr int most = (1 << 24) - 1;
    auto pieces = [&](const Range& r) {
        const AttnPlan<BM, BN> p(A, r.lq, r.lk);
        return min(p.tiles * p.chunks, most);
    };
    const int xcd = block & 7, slot = block >> 3, share = 8 / A.classes;
    const int idx = slot * share + xcd / A.classes;
    Range mine = {0, 0, 0, 0};
    int seq = lane;   // whose range that is, behind `base`
    int per_head, sum = 0;  // pieces to a key head; of the sequences up to this lane's (the first 64)
    if (A.cu_q) {
        if (lane < A.batch) {
            mine = range(lane);
            sum = pieces(mine);
        }
        if (BM > 32 && A.batch <= 64) {
            int rank = lane;
            if (lane < A.batch) {
                rank = 0;
                for (int i = 0; i < A.batch; ++i) {
                    const int other = __builtin_amdgcn_readlane(mine.lk, i);
                    rank += other > mine.lk || (other == mine.lk && i < lane);
                }
            }
            auto move = [&](int& v) { v = __builtin_amdgcn_ds_permute(rank * 4, v); };
            move(mine.q0);
            move(mine.lq);
            move(mine.k0);
            move(mine.lk);
            move(sum);
            move(seq);
        }
        sum = wave_scan(sum, lane, A.batch);
        per_head = __builtin_amdgcn_readlane(sum, min(A.batch, 64) - 1);
        if (A.batch > 64) {
            int n = 0;
            for (int s = 64 + lane; s < A.batch; s += 64) n = min(n + pieces(range(s)), most);
            per_head += __builtin_amdgcn_readlane(wave_scan(n, lane, 64), 63);
        }
    } else {
        per_head = A.batch * A.pieces;
    }
    if (per_head == 0) return false;
    const int hi = A.kv_heads == A.classes ? (idx < per_head ? 0 : 1) : sgpr(idx / per_head);
    if (hi >= A.kv_heads / A.classes) return false;
    w.kvh = xcd % A.classes + A.classes * hi;
    int r = idx - hi * per_head;
    if (A.cu_q) {
        int before = 0, base = 0;  // pieces before lane 0's sequence, and that sequence
        uint64_t over = __ballot(lane < A.batch && sum > r);
        while (over == 0) {
            before += __builtin_amdgcn_readlane(sum, 63);
            base += 64;
            if (base >= A.batch) return false;  // (the offsets have changed meanwhile)
            sum = 0;
            if (base + lane < A.batch) {
                mine = range(base + lane);
                sum = pieces(mine);
            }
            sum = wave_scan(sum, lane, 64);
            over = __ballot(before + sum > r);
        }
        const int l = __builtin_ctzll(over);
        if (l > 0) before += __builtin_amdgcn_readlane(sum, l - 1);
        r = sgpr(r - before);
        w.seq = base + __builtin_amdgcn_readlane(seq, l);
        w.q0 = __builtin_amdgcn_readlane(mine.q0, l);
        w.lq = __builtin_amdgcn_readlane(mine.lq, l);
        w.k0 = __builtin_amdgcn_readlane(mine.k0, l);
        w.lk = __builtin_amdgcn_readlane(mine.lk, l);
    } else {
        w.seq = A.batch == 1 ? 0 : sgpr(r / A.pieces);
        r -= w.seq * A.pieces;
        w.q0 = w.seq * A.len_q;
        w.lq = A.len_q;
        w.k0 = 0;
        w.lk = A.len_k;
    }
    const AttnPlan<BM, BN> p(A, w.lq, w.lk);
    const int tiles = sgpr(p.tiles);
    w.chunks = sgpr(p.chunks);
    w.chunk = w.chunks == 1 ? 0 : sgpr(r / tiles);
    w.tile = tiles - 1 - (r - w.chunk * tiles);
    return true;
}

// ---- launchers --------------------------------------------------------------
lynx_status launch_qk_rotary(const lynx_rotary& d, hipStream_t stream);

lynx_status launch_attn_tile(const AttnArgs& a, int grid, hipStream_t stream);
lynx_status launch_attn_wide(const AttnArgs& a, int grid, hipStream_t stream);
lynx_status launch_attn_few(const AttnArgs& a, int grid, hipStream_t stream);
lynx_status launch_attn_near(const AttnArgs& a, int grid, hipStream_t stream);
// `tile` (not causal) and `few` side by side, in one launch
lynx_status launch_attn_pair(const AttnArgs& tile, int tile_grid, const AttnArgs& few, int few_grid,
                             hipStream_t stream);
lynx_status launch_attn_join(const AttnArgs& a, int prefix_slots, hipStream_t stream);

}  // namespace lynx
