// C ABI of rotary positions and attention: argument validation, the choice of kernel and of
// the split of keys, workspace layout and dispatch.  Defined in lynx.h.
#include <cmath>
#include <initializer_list>
#include <numeric>

#include "lynx_attn.h"
#include "lynx_debug.h"

namespace lynx {
namespace {

constexpr int64_t kMaxRotaryTokens = int64_t(1) << 24, kMaxHeads = 1024;
constexpr int64_t kMaxAttnTokens = int64_t(1) << 26, kMaxBatch = int64_t(1) << 16;
constexpr int64_t kMaxTokenStride = int64_t(1) << 24;  // 64 rows stay below 2^31 bytes
constexpr int64_t kMaxQueryRows = int64_t(1) << 30;

bool all16(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!aligned16(p)) return false;
    return true;
}

bool strides_ok(std::initializer_list<int64_t> ss) {
    for (int64_t s : ss)
        if (s < 0 || s % 8 != 0) return false;
    return true;
}

lynx_status validate_rotary(const lynx_rotary& d, bool* noop) {
    *noop = false;
    if (d.head_dim < 8 || d.head_dim > 256 || d.head_dim % 8 != 0) return LYNX_ERR_SHAPE;
    if (d.tokens < 0 || d.tokens > kMaxRotaryTokens) return LYNX_ERR_SHAPE;
    if (d.q_heads < 1 || d.q_heads > kMaxHeads || d.k_heads < 0 || d.k_heads > kMaxHeads)
        return LYNX_ERR_SHAPE;
    if (d.tokens * (d.q_heads + d.k_heads) >= (int64_t(1) << 31)) return LYNX_ERR_SHAPE;
    if (d.axes < 1 || d.axes > 4) return LYNX_ERR_SHAPE;
    int64_t R = 0;
    for (int i = 0; i < d.axes; ++i) {
        if (d.axis_dims[i] < 2 || d.axis_dims[i] > 256 || d.axis_dims[i] % 2 != 0) return LYNX_ERR_SHAPE;
        R += d.axis_dims[i];
    }
    if (R > d.head_dim) return LYNX_ERR_SHAPE;
    if (!(d.theta > 0.0) || !std::isfinite(d.theta)) return LYNX_ERR_SHAPE;
    if (d.pairs != LYNX_PAIRS_ADJACENT && d.pairs != LYNX_PAIRS_HALVES) return LYNX_ERR_SHAPE;
    if (d.ladder != LYNX_LADDER_AXIS && d.ladder != LYNX_LADDER_JOINT) return LYNX_ERR_SHAPE;
    if (d.norm != LYNX_NORM_NONE && d.norm != LYNX_NORM_RMS) return LYNX_ERR_SHAPE;
    if (!(d.eps >= 0.f)) return LYNX_ERR_SHAPE;
    if (!strides_ok({d.q_stride, d.q_head_stride, d.q_out_stride, d.q_out_head_stride}))
        return LYNX_ERR_SHAPE;
    if (d.k_heads > 0 && !strides_ok({d.k_stride, d.k_head_stride, d.k_out_stride, d.k_out_head_stride}))
        return LYNX_ERR_SHAPE;
    if (d.tokens == 0) {
        *noop = true;
        return LYNX_OK;
    }
    if (!d.q || !d.q_out || !d.positions) return LYNX_ERR_NULL;
    if (d.k_heads > 0 ? (!d.k || !d.k_out) : (d.k || d.k_out || d.k_weight)) return LYNX_ERR_NULL;
    if (d.norm == LYNX_NORM_NONE && (d.q_weight || d.k_weight)) return LYNX_ERR_NULL;
    if (!all16({d.q, d.k, d.q_weight, d.k_weight, d.positions, d.q_out, d.k_out})) return LYNX_ERR_ALIGN;
    return LYNX_OK;
}

// Sizes alone: what the workspace depends on.
bool attn_sizes_ok(const lynx_attn& d) {
    if (d.head_dim < 8 || d.head_dim > 128 || d.head_dim % 8 != 0) return false;
    if (d.kv_heads < 1 || d.heads < 1 || d.heads > kMaxHeads || d.heads % d.kv_heads != 0) return false;
    if (d.batch < 1 || d.batch > kMaxBatch) return false;
    for (int64_t t : {d.tokens_q, d.tokens_k, d.prefix_tokens})
        if (t < 0 || t > kMaxAttnTokens) return false;
    return d.tokens_q * d.heads < kMaxQueryRows;
}

lynx_status validate_attn(const lynx_attn& d, bool* noop) {
    *noop = false;
    if (!attn_sizes_ok(d)) return LYNX_ERR_SHAPE;
    if (!(d.scale > 0.f) || !std::isfinite(d.scale)) return LYNX_ERR_SHAPE;
    if ((d.cu_q != nullptr) != (d.cu_k != nullptr)) return LYNX_ERR_NULL;
    if (!d.cu_q && (d.tokens_q % d.batch != 0 || d.tokens_k % d.batch != 0)) return LYNX_ERR_SHAPE;
    if (!strides_ok({d.q_stride, d.q_head_stride, d.k_stride, d.k_head_stride, d.v_stride,
                     d.v_head_stride, d.out_stride, d.out_head_stride}))
        return LYNX_ERR_SHAPE;
    if (!d.cu_q && !strides_ok({d.q_batch_stride, d.k_batch_stride, d.v_batch_stride, d.out_batch_stride}))
        return LYNX_ERR_SHAPE;
    auto key_stride_ok = [&](int64_t s) { return s >= d.head_dim && s < kMaxTokenStride; };
    if (d.tokens_k > 0 && (!key_stride_ok(d.k_stride) || !key_stride_ok(d.v_stride))) return LYNX_ERR_SHAPE;
    if (d.prefix_tokens > 0 &&
        (!key_stride_ok(d.prefix_k_stride) || !key_stride_ok(d.prefix_v_stride) ||
         !strides_ok({d.prefix_k_stride, d.prefix_v_stride, d.prefix_k_head_stride, d.prefix_v_head_stride})))
        return LYNX_ERR_SHAPE;
    if (d.tokens_q == 0) {
        *noop = true;
        return LYNX_OK;
    }
    if (!d.q || !d.out) return LYNX_ERR_NULL;
    if (d.tokens_k > 0 && (!d.k || !d.v)) return LYNX_ERR_NULL;
    if (d.prefix_tokens > 0 ? (!d.prefix_k || !d.prefix_v) : (d.prefix_k || d.prefix_v)) return LYNX_ERR_NULL;
    if (!all16({d.q, d.k, d.v, d.prefix_k, d.prefix_v, d.out})) return LYNX_ERR_ALIGN;
    for (const void* p : {static_cast<const void*>(d.cu_q), static_cast<const void*>(d.cu_k),
                          static_cast<const void*>(d.lse)})
        if ((reinterpret_cast<uintptr_t>(p) & 3u) != 0) return LYNX_ERR_ALIGN;
    return LYNX_OK;
}

// One launch over keys: which kernel, and how keys are cut.
struct Pass {
    bool few;
    int chunk_tiles, chunk_max;  // as in AttnArgs; chunk_max 1: not cut
    int64_t grid;
};

struct Plan {
    bool apart;       // the prefix in a pass of its own
    Pass prefix, own;
    int slots;        // of a row's partial results, 0: none
    size_t o, ml, n, total;  // workspace
};

constexpr int kUnits = 256;

// rows: query rows to a key head, over all sequences; keys: of all sequences together, shared:
// keys that each sequence has besides
Pass plan_pass(int64_t batch, int64_t rows, int64_t keys, int64_t shared, int64_t kv_heads, bool ragged) {
    Pass p;
    const int64_t mean_rows = (rows + batch - 1) / batch;
    p.few = mean_rows <= 32;
    const int64_t bm = p.few ? 32 : 128, bn = p.few ? 128 : 64;
    const int64_t tiles = batch * ((mean_rows + bm - 1) / bm) * kv_heads;     // of rows, about
    const int64_t kt = ((keys + batch - 1) / batch + shared + bn - 1) / bn;   // key tiles of one
    const int64_t want = p.few ? 2 * kUnits : 2 * kUnits;
    int64_t chunks = tiles >= want ? 1 : want / tiles;
    const int64_t least = p.few ? 2 : 4;
    chunks = std::max<int64_t>(1, std::min(chunks, kt / least));
    int64_t per = std::max<int64_t>(1, (kt + chunks - 1) / chunks);
    // sequences longer than the mean have more chunks
    const int64_t all = (keys + shared + bn - 1) / bn;
    int64_t top = ragged ? (all + per - 1) / per : (kt + per - 1) / per;
    if (ragged && p.few && top > 1) {
        // one long sequence among short ones is cut too
    } else if (chunks == 1) {
        top = 1;
    }
    top = std::max<int64_t>(1, std::min<int64_t>(top, 64));
    // no more than 256 MB of partial results for the sake of uneven lengths
    top = std::min(top, std::max(chunks, (int64_t(1) << 28) / (rows * kv_heads * 528)));
    p.chunk_tiles = int(per);
    p.chunk_max = int(top);
    const int64_t most_tiles = (ragged ? rows / bm + batch : batch * ((mean_rows + bm - 1) / bm));
    int64_t items = most_tiles * top;  // to a key head, at most
    const int64_t classes = std::gcd<int64_t>(kv_heads, 8), share = 8 / classes;
    int64_t grid = 8 * ((kv_heads / classes * items + share - 1) / share);
    if (top > 1) grid = std::min<int64_t>(grid, p.few ? kUnits : 2 * kUnits);
    p.grid = std::min<int64_t>(grid, int64_t(1) << 22);
    return p;
}

Plan make_plan(const lynx_attn& d, bool ragged) {
    Plan P = {};
    const int64_t group = d.heads / d.kv_heads, rows = d.tokens_q * group;
    P.apart = d.prefix_tokens > 0 && d.batch > 1 && rows / d.batch < 128;
    P.own = plan_pass(d.batch, rows, d.tokens_k, P.apart ? 0 : d.prefix_tokens, d.kv_heads, ragged);
    int slots = P.own.chunk_max > 1 ? P.own.chunk_max : 0;
    if (P.apart) {
        P.prefix = plan_pass(1, rows, d.prefix_tokens, 0, d.kv_heads, false);
        slots = P.own.chunk_max + P.prefix.chunk_max;
    }
    P.slots = slots;
    if (slots > 0) {
        const size_t r = size_t(d.tokens_q) * size_t(d.heads), s = size_t(slots);
        P.o = 0;
        P.ml = round_up256(r * s * size_t(d.head_dim) * 4);
        P.n = P.ml + round_up256(r * s * 16);
        P.total = P.n + round_up256(r * 4);
    }
    return P;
}

}  // namespace
}  // namespace lynx

using namespace lynx;

extern "C" {

lynx_status lynx_qk_rotary(const lynx_rotary* rotary, lynx_stream_t stream) {
    if (!rotary) return LYNX_ERR_NULL;
    const lynx_rotary d = *rotary;
    bool noop = false;
    lynx_status st = validate_rotary(d, &noop);
    if (st != LYNX_OK || noop) return st;
    st = check_device();
    if (st != LYNX_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return debug_sync(launch_qk_rotary(d, s), s);
}

size_t lynx_attention_workspace_bytes(const lynx_attn* attn) {
    if (!attn || !attn_sizes_ok(*attn)) return 0;
    return make_plan(*attn, attn->cu_q != nullptr).total;
}

lynx_status lynx_attention(const lynx_attn* attn, void* workspace, size_t workspace_bytes,
                           lynx_stream_t stream) {
    if (!attn) return LYNX_ERR_NULL;
    const lynx_attn d = *attn;
    bool noop = false;
    lynx_status st = validate_attn(d, &noop);
    if (st != LYNX_OK || noop) return st;
    const Plan P = make_plan(d, d.cu_q != nullptr);
    if (P.total > 0) {
        if (!workspace || workspace_bytes < P.total) return LYNX_ERR_WORKSPACE;
        if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return LYNX_ERR_ALIGN;
    }
    st = check_device();
    if (st != LYNX_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);

    AttnArgs a = {};
    a.q = d.q;
    a.k = d.k;
    a.v = d.v;
    a.cu_q = d.cu_q;
    a.cu_k = d.cu_k;
    a.out = d.out;
    a.lse = d.lse;
    char* ws = static_cast<char*>(workspace);
    if (P.slots > 0) {
        a.part_o = reinterpret_cast<float*>(ws + P.o);
        a.part_ml = reinterpret_cast<float4*>(ws + P.ml);
        a.part_n = reinterpret_cast<int*>(ws + P.n);
    }
    a.q_b = d.q_batch_stride;
    a.q_t = d.q_stride;
    a.q_h = d.q_head_stride;
    a.o_b = d.out_batch_stride;
    a.o_t = d.out_stride;
    a.o_h = d.out_head_stride;
    a.k_b = d.k_batch_stride;
    a.k_t = d.k_stride;
    a.k_h = d.k_head_stride;
    a.v_b = d.v_batch_stride;
    a.v_t = d.v_stride;
    a.v_h = d.v_head_stride;
    a.batch = int(d.batch);
    a.heads = int(d.heads);
    a.kv_heads = int(d.kv_heads);
    a.group = int(d.heads / d.kv_heads);
    a.D = int(d.head_dim);
    a.tokens_q = int(d.tokens_q);
    a.tokens_k = int(d.tokens_k);
    a.len_q = int(d.tokens_q / d.batch);
    a.len_k = int(d.tokens_k / d.batch);
    a.addr_len = d.cu_q ? INT32_MAX : a.len_q;
    a.slots = P.slots;
    a.classes = int(std::gcd<int64_t>(d.kv_heads, 8));
    a.c = d.scale * kLog2e;
    a.causal = d.causal != 0;

    auto run = [&](const AttnArgs& args, const Pass& p) {
        return p.few ? launch_attn_few(args, int(p.grid), s) : launch_attn_tile(args, int(p.grid), s);
    };
    if (P.apart) {
        AttnArgs p = a;
        p.k = d.prefix_k;
        p.v = d.prefix_v;
        p.cu_q = p.cu_k = nullptr;
        p.k_b = p.v_b = 0;
        p.k_t = d.prefix_k_stride;
        p.k_h = d.prefix_k_head_stride;
        p.v_t = d.prefix_v_stride;
        p.v_h = d.prefix_v_head_stride;
        p.batch = 1;
        p.len_q = a.tokens_q;
        p.tokens_k = p.len_k = int(d.prefix_tokens);
        p.causal = 0;
        p.force_part = 1;
        p.chunk_tiles = P.prefix.chunk_tiles;
        p.chunk_max = P.prefix.chunk_max;
        st = run(p, P.prefix);
        if (st != LYNX_OK) return st;
        a.slot0 = P.prefix.chunk_max;
        a.force_part = 1;
    } else {
        a.pk = d.prefix_k;
        a.pv = d.prefix_v;
        a.pk_t = d.prefix_k_stride;
        a.pk_h = d.prefix_k_head_stride;
        a.pv_t = d.prefix_v_stride;
        a.pv_h = d.prefix_v_head_stride;
        a.prefix = int(d.prefix_tokens);
    }
    a.chunk_tiles = P.own.chunk_tiles;
    a.chunk_max = P.own.chunk_max;
    st = run(a, P.own);
    if (st != LYNX_OK) return st;
    if (P.slots > 0) {
        st = launch_attn_join(a, a.slot0, s);
        if (st != LYNX_OK) return st;
    }
    return debug_sync(st, s);
}

}  // extern "C"
