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

// Arguments of an attention kernel.  Query rows of one sequence and key head are numbered
// token * group + head in group, so that the heads that share a key head share its tiles.
//
// Keys are cut into tiles (the prefix' tiles first, then the sequence's own), tiles into
// chunks of at least chunk_tiles, at most chunk_max of them to a sequence.  Work is the list
// of (sequence, key head, row tile, chunk).  Where slots > 0 a chunk's result goes to the
// partial sums: row's slot slot0 + chunk, part_n[row] chunks; lynx_attn_join adds them up.  A
// sequence of one chunk goes straight to out, unless force_part.
struct AttnArgs {
    const uint16_t *q, *k, *v, *pk, *pv;
    const int *cu_q, *cu_k;
    uint16_t* out;
    float* lse;
    float* part_o;    // [row][slot][D]
    float4* part_ml;  // [row][slot]: m in powers of two, l, l of unrounded weights (with lse)
    int* part_n;      // [row]
    int64_t q_b, q_t, q_h, o_b, o_t, o_h;
    int64_t k_b, k_t, k_h, v_b, v_t, v_h, pk_t, pk_h, pv_t, pv_h;
    int batch, heads, kv_heads, group, D;
    int tokens_q, tokens_k, prefix;
    int len_q, len_k;    // uniform form: tokens of a sequence
    int addr_len;        // tokens of q and out that are q_t apart
    int slots, slot0, force_part, chunk_tiles, chunk_max;
    int classes;         // gcd(kv_heads, 8)
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

// inclusive sum over the lanes of a wave
__device__ __forceinline__ int wave_scan(int v, int lane) {
#pragma unroll
    for (int d = 1; d < 64; d *= 2) {
        const int o = __shfl_up(v, d);
        if (lane >= d) v += o;
    }
    return v;
}

// Row tiles and chunks of a sequence.
template <int BM, int BN>
struct AttnPlan {
    int tiles, chunks, per;  // per: key tiles of a chunk
    __device__ __forceinline__ AttnPlan(const AttnArgs& A, int lq, int lk) {
        tiles = (lq * A.group + BM - 1) / BM;
        const int kt = (A.prefix + BN - 1) / BN + (lk + BN - 1) / BN;
        if (A.chunk_max == 1) {
            per = max(kt, 1);
            chunks = 1;
        } else {
            per = max(A.chunk_tiles, (kt + A.chunk_max - 1) / A.chunk_max);
            chunks = max(1, (kt + per - 1) / per);
        }
    }
};

// Walks the work of one workgroup.  Workgroups of one XCD (their number mod 8) take the
// same key heads, one after the other, so that its L2 holds the keys and values that its
// workgroups read; where there are fewer key heads than XCDs several share a head.  Within a
// head sequences follow one another, and a sequence's row tiles come last tile first: under a
// causal mask these have the most keys, and the light ones fill the end.
template <int BM, int BN>
struct AttnWork {
    int idx, step, per_head, heads;
    const AttnArgs& A;
    int lane;

    __device__ __forceinline__ void range(int s, int& q0, int& lq, int& k0, int& lk) const {
        const int qa = clampi(A.cu_q[s], 0, A.tokens_q), qb = clampi(A.cu_q[s + 1], qa, A.tokens_q);
        const int ka = clampi(A.cu_k[s], 0, A.tokens_k), kb = clampi(A.cu_k[s + 1], ka, A.tokens_k);
        q0 = qa;
        lq = qb - qa;
        k0 = ka;
        lk = kb - ka;
    }
    __device__ __forceinline__ int count(int s) const {
        if (s >= A.batch) return 0;
        int q0, lq, k0, lk;
        range(s, q0, lq, k0, lk);
        const AttnPlan<BM, BN> p(A, lq, lk);
        return p.tiles * p.chunks;
    }

    __device__ __forceinline__ explicit AttnWork(const AttnArgs& a) : A(a) {
        lane = threadIdx.x & 63;
        if (A.cu_q) {
            int n = 0;
            for (int s = lane; s < A.batch; s += 64) n += count(s);
            per_head = __builtin_amdgcn_readlane(wave_scan(n, lane), 63);
        } else {
            const AttnPlan<BM, BN> p(A, A.len_q, A.len_k);
            per_head = A.batch * p.tiles * p.chunks;
        }
        const int xcd = int(blockIdx.x) & 7, slot = int(blockIdx.x) >> 3, share = 8 / A.classes;
        idx = slot * share + xcd / A.classes;
        step = (int(gridDim.x) >> 3) * share;  // the grid is a multiple of 8
        heads = A.kv_heads / A.classes;
    }

    // the next piece; false at the end.  Uniform over the workgroup.
    __device__ __forceinline__ bool next(AttnItem& w) {
        if (per_head == 0) return false;
        const int hi = sgpr(idx / per_head);
        if (hi >= heads) return false;
        int r = idx - hi * per_head;
        idx += step;
        w.kvh = (int(blockIdx.x) & 7) % A.classes + A.classes * hi;
        if (A.cu_q) {
            int before = 0, s = 0;
            for (int base = 0; base < A.batch; base += 64) {
                const int n = count(base + lane);
                const int sum = wave_scan(n, lane);
                const uint64_t over = __ballot(before + sum > r);
                if (over) {
                    const int l = __builtin_ctzll(over);
                    s = base + l;
                    before += __builtin_amdgcn_readlane(sum, l) - __builtin_amdgcn_readlane(n, l);
                    break;
                }
                before += __builtin_amdgcn_readlane(sum, 63);
            }
            r = sgpr(r - before);
            w.seq = sgpr(s);
            int q0, lq, k0, lk;
            range(w.seq, q0, lq, k0, lk);
            w.q0 = sgpr(q0);
            w.lq = sgpr(lq);
            w.k0 = sgpr(k0);
            w.lk = sgpr(lk);
            const AttnPlan<BM, BN> p(A, w.lq, w.lk);
            w.chunks = p.chunks;
            w.chunk = sgpr(r / p.tiles);
            w.tile = p.tiles - 1 - (r - w.chunk * p.tiles);
        } else {
            const AttnPlan<BM, BN> p(A, A.len_q, A.len_k);
            const int per = p.tiles * p.chunks;
            const int s = sgpr(r / per);
            r -= s * per;
            w.seq = s;
            w.q0 = s * A.len_q;
            w.lq = A.len_q;
            w.k0 = int64_t(s) * A.len_k;
            w.lk = A.len_k;
            w.chunks = p.chunks;
            w.chunk = sgpr(r / p.tiles);
            w.tile = p.tiles - 1 - (r - w.chunk * p.tiles);
        }
        return true;
    }
};

// ---- launchers --------------------------------------------------------------
lynx_status launch_qk_rotary(const lynx_rotary& d, hipStream_t stream);

lynx_status launch_attn_tile(const AttnArgs& a, int grid, hipStream_t stream);
lynx_status launch_attn_few(const AttnArgs& a, int grid, hipStream_t stream);
lynx_status launch_attn_join(const AttnArgs& a, int prefix_slots, hipStream_t stream);

}  // namespace lynx
