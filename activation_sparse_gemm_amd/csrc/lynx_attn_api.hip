// C ABI of rotary positions and attention: argument validation, the choice of kernel and of
// the split of keys, workspace layout and dispatch.  Defined in lynx.h.
#include <algorithm>
#include <cmath>
#include <initializer_list>
#include <numeric>

#include "lynx_attn.h"
#include "lynx_debug.h"

namespace lynx {
namespace {

constexpr int64_t kMaxRotaryTokens = int64_t(1) << 24, kMaxHeads = 1024;
constexpr int64_t kMaxAttnTokens = int64_t(1) << 26, kMaxBatch = int64_t(1) << 16;
constexpr int64_t kMaxTokenStride = int64_t(1) << 23;  // a tile's 128 rows stay below 2^31 bytes
constexpr int64_t kMaxQueryRows = int64_t(1) << 30;
constexpr int64_t kMaxPairs = int64_t(1) << 21;  // sequences times key heads: a launch has below 2^32 threads

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
    if (!(d.theta > 0.0) || !std::isnormal(d.theta)) return LYNX_ERR_SHAPE;  // (1 / theta is finite)
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
    if (d.batch < 1 || d.batch > kMaxBatch || d.batch * d.kv_heads > kMaxPairs) return false;
    for (int64_t t : {d.tokens_q, d.tokens_k, d.prefix_tokens})
        if (t < 0 || t > kMaxAttnTokens) return false;
    return d.tokens_q * d.heads < kMaxQueryRows;
}

lynx_status validate_attn(const lynx_attn& d, bool* noop) {
    *noop = false;
    if (!attn_sizes_ok(d)) return LYNX_ERR_SHAPE;
    if (!(d.scale > 0.f) || !(d.scale < 0x1p127f)) return LYNX_ERR_SHAPE;  // (log2(e) times it is finite)
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
enum class Kernel { few, near, tile, wide };
struct Pass {
    Kernel kernel;
    int chunk_tiles, chunk_max;  // as in AttnArgs; chunk_max 1: not cut
    int64_t grid;
    int shares;  // near: of a sequence's rows
};

struct Plan {
    bool apart;       // the prefix in a pass of its own
    Pass prefix, own;
    int slots;        // of a row's partial results, 0: none
    size_t o, ml, n, total;  // workspace
};

constexpr int kUnits = 256;

// Row tiles and chunks that the kernel of pass p makes of a sequence of lq queries and lk keys; as its
// workgroups work them out.
struct Cut {
    int tiles, chunks;
};
Cut cut_of(const Pass& p, int group, int prefix, int64_t D, int lq, int lk) {
    AttnArgs a = {};
    a.group = group;
    a.prefix = prefix;
    a.chunk_tiles = p.chunk_tiles;
    a.chunk_max = p.chunk_max;
    auto of = [](auto plan) { return Cut{plan.tiles, plan.chunks}; };
    const bool small = D <= 64;  // (tiles of keys are 128 then)
    if (p.kernel == Kernel::few) return of(AttnPlan<32, 128>(a, lq, lk));
    if (p.kernel == Kernel::tile)
        return small ? of(AttnPlan<128, 128>(a, lq, lk)) : of(AttnPlan<128, 64>(a, lq, lk));
    return small ? of(AttnPlan<256, 128>(a, lq, lk)) : of(AttnPlan<256, 64>(a, lq, lk));
}

// Which kernel takes a pass, and into how many chunks it cuts the keys.  rows: query rows to a
// key head, over all sequences; keys: of all sequences together; shared: keys that each sequence has
// besides; seen: the share of the keys that a mask leaves; joined: whether the join runs anyway;
// beside: workgroups of the few-row kernel that run side by side with this pass.
Pass plan_pass(int64_t batch, int64_t rows, int64_t keys, int64_t shared, int64_t kv_heads, int64_t D,
               bool ragged, double seen, bool joined, int64_t beside) {
    Pass p = {};
    constexpr int64_t kMaxPartial = int64_t(1) << 28;
    const int64_t mean_rows = (rows + batch - 1) / batch, row_bytes = kv_heads * rows * (D * 4 + 16);
    auto tiles_of = [&](int64_t m) { return batch * ((mean_rows + m - 1) / m) * kv_heads; };
    // per: key tiles of a chunk; top: the most chunks of a sequence, and no more than 256 MB of
    // partial results for the sake of uneven lengths
    auto finish = [&](Kernel kernel, int64_t bm, int64_t bn, int64_t per, int64_t chunks) {
        const int64_t most = (keys + bn - 1) / bn + (shared + bn - 1) / bn;  // were all in one sequence
        int64_t top = ragged && chunks > 0 ? (most + per - 1) / per : chunks;
        top = std::min(top, std::max(chunks, kMaxPartial / row_bytes));
        top = std::max<int64_t>(1, std::min<int64_t>(top, kMaxChunks));
        p.kernel = kernel;
        p.chunk_tiles = int(per);
        p.chunk_max = int(top);
        // The length of the work list, at most: a sequence has one row tile, and one more for
        // every bm rows, and its chunks hold `per` key tiles each but the last one
        int64_t items = tiles_of(bm) / kv_heads * top;
        if (ragged) {
            const int64_t all = keys / bn + batch * (1 + (shared + bn - 1) / bn);
            items = (rows / bm + batch) * top;
            items = std::min(items, all / per + batch + rows / bm * (kernel == Kernel::few ? 1 : top));
        }
        const int64_t classes = std::gcd<int64_t>(kv_heads, 8), share = 8 / classes;
        p.grid = 8 * ((kv_heads / classes * items + share - 1) / share);
    };
    if (mean_rows <= 32) {
        // Bound by the keys' bytes: two workgroups to a unit, and no fewer than that.  Sequences
        // of different lengths are cut into four times as many chunks of one size, so that the
        // units end together: 32 tokens on caches of 17 .. 16400 keys 212 us, without 229.
        const int64_t kt = std::max<int64_t>(1, ((keys + batch - 1) / batch + shared + 127) / 128);
        const int64_t tiles = tiles_of(32), want = (ragged && batch > 1 ? 8 : 2) * kUnits;
        // (at least 4 tiles, 8 with all 32 rows: partial results are then an eighth of the keys)
        int64_t per = std::max({int64_t(4), mean_rows / 4, (tiles * kt + want - 1) / want});
        const int64_t chunks = (kt + per - 1) / per;
        if (!ragged || batch == 1) per = (kt + chunks - 1) / chunks;
        finish(Kernel::few, 32, 128, per, chunks);
        return p;
    }
    // By estimated time.  A compute unit takes, per tile of keys (128 channels: 64 keys; up to 64
    // channels: 128):
    //   128 rows (tile)  1.03 us (1.2), two workgroups to a unit taking as long as one after
    //                    the other: 16384 x 16384 x 8 heads 1058 us
    //   256 rows (wide)  1.92 us (2.28), one workgroup to a unit: 985 us
    // and 5 us for what comes before and after.  Under a causal mask row tiles differ, and units
    // that have light ones take more of them; but the heaviest takes its time.  Cutting needs
    // the join: 4 us, and its bytes, which are written and read at 4 TB/s.
    const int64_t bn = D <= 64 ? 128 : 64;
    const int64_t kt = ((keys + batch - 1) / batch + shared + bn - 1) / bn;
    double best = 0.0;
    double besides = 0.0;  // what the best's row tiles take besides, as the kernel for few keys sees it
    // (packed sequences differ: the 256-row tiles of a long one end late)
    for (int wide = 0; wide < (ragged && batch > 1 ? 1 : 2); ++wide) {
        const int64_t bm = wide ? 256 : 128, tiles = tiles_of(bm);
        const double step = wide ? (D <= 64 ? 2.28 : 1.92) : (D <= 64 ? 1.20 : 1.03);
        for (int64_t chunks = 1; chunks <= kMaxChunks && (chunks == 1 || chunks * 2 <= kt + 1); ++chunks) {
            const int64_t per = std::max<int64_t>(1, (kt + chunks - 1) / chunks), items = tiles * chunks;
            if (chunks > 1 && row_bytes * chunks > kMaxPartial) break;
            double us = double((items + kUnits - 1) / kUnits) * double(per) * step;
            if (seen < 1.0)
                us = std::max(double(items) / kUnits * double(per) * seen * step,
                              double(per) * step * (wide || items <= kUnits ? 1.0 : 1.6));
            if (joined) us += double(row_bytes * chunks) * 2.0 / 4.0e6;
            else if (chunks > 1) us += 4.0 + double(row_bytes * chunks) * 2.0 / 4.0e6;
            // The few-row kernel runs beside the tile kernel, but after the wide one.  Units have room
            // for two workgroups: where that is enough for the few-row kernel's alone, those
            // that have to wait for a tile end late (48 tokens on a prefix of 8192: 10 chunks
            // 31 us, 16 39; 48 x 4 on 4096: wide 52, tile 35).
            const int64_t over = items + beside - 2 * kUnits;
            if (beside > 0 && wide) us += 14.0;
            else if (beside > 0 && beside <= 2 * kUnits && over > 0) us += 14.0 * std::min(1.0, double(over) / 256.0);
            if (best == 0.0 || us < best) {
                best = us;
                besides = double((items + kUnits - 1) / kUnits) * (wide ? 7.0 : 3.5);
                finish(wide ? Kernel::wide : Kernel::tile, bm, bn, per, chunks == 1 ? 0 : chunks);
            }
            if (items >= 8 * kUnits) break;
        }
    }
    // Few keys, the same for all sequences: the kernel that holds them all in LDS.  To it, 256 rows
    // and a tile of keys are 2.3 us, and there are 5 us besides for a workgroup; to the others, 3.5 us
    // (wide: 7) besides for each row tile that a unit takes.  4608 x 256 x 24 heads 26 us (34), 20000 x 300
    // x 28 heads 120 (179); on the other side 1024 x 300 x 24 heads 17 us (12, and that is taken).
    if (!ragged && seen == 1.0 && shared == 0 && !joined && kt >= 1 && kt <= kNearTiles) {
        const int64_t pairs = batch * kv_heads, tiles = (mean_rows + 31) / 32;
        best += besides;
        for (int64_t r = 1; r <= 4; ++r) {  // workgroups to a unit
            int64_t shares = std::max<int64_t>(1, std::min(r * kUnits / pairs, (tiles + 7) / 8));
            const int64_t steps = ((tiles + shares - 1) / shares + 7) / 8;  // of a wave, for each tile of keys
            shares = (tiles + 8 * steps - 1) / (8 * steps);                 // the fewest for that
            const double us = double((pairs * shares + kUnits - 1) / kUnits) *
                              (5.0 + double(steps) * double(kt) * 2.3);
            if (us >= best) continue;
            best = us;
            p.kernel = Kernel::near;
            p.chunk_tiles = int(kt);
            p.chunk_max = 1;
            p.shares = int(shares);
            p.grid = pairs * shares;
        }
    }
    return p;
}

Plan make_plan(const lynx_attn& d, bool ragged) {
    Plan P = {};
    if (d.tokens_q == 0) return P;
    const int64_t group = d.heads / d.kv_heads, rows = d.tokens_q * group;
    // A prefix is worked on once for all sequences where their rows alone do not fill row tiles
    // (and where the partial results of both passes are not past a GiB)
    P.apart = d.prefix_tokens > 0 && d.batch > 1 && rows / d.batch < 128 &&
              d.tokens_q * d.heads * (d.head_dim * 4 + 16) <= (int64_t(1) << 29);
    const int64_t shared = P.apart ? 0 : d.prefix_tokens;
    double seen = 1.0;
    if (d.causal) {
        const double keys = double(d.tokens_k) + double(d.batch) * double(shared);
        if (keys > 0.0) seen = std::max(0.5, 1.0 - 0.5 * double(d.tokens_q) / keys);
    }
    P.own = plan_pass(d.batch, rows, d.tokens_k, shared, d.kv_heads, d.head_dim, ragged, seen, P.apart, 0);
    int slots = P.own.chunk_max > 1 ? P.own.chunk_max : 0;
    if (P.apart) {
        const int64_t pairs = P.own.kernel == Kernel::few ? d.batch * d.kv_heads : 0;
        P.prefix = plan_pass(1, rows, d.prefix_tokens, 0, d.kv_heads, d.head_dim, false, 1.0, true, pairs);
        // The join reads as many slots of every row as this says, so it has to be what is written:
        // 547 tiles in at most 128 chunks are 110 of 5.
        P.prefix.chunk_max =
            cut_of(P.prefix, int(group), 0, d.head_dim, int(d.tokens_q), int(d.prefix_tokens)).chunks;
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
    a.addr_len = d.cu_q || d.batch == 1 ? 0 : a.len_q;
    a.group_shift = (a.group & (a.group - 1)) == 0 ? __builtin_ctz(unsigned(a.group)) : -1;
    a.slots = P.slots;
    a.classes = int(std::gcd<int64_t>(d.kv_heads, 8));
    a.c = d.scale * kLog2e;
    a.causal = d.causal != 0;

    // a pass' arguments, and its launch
    auto cut = [&](AttnArgs& args, const Pass& p) {
        args.chunk_tiles = p.chunk_tiles;
        args.chunk_max = p.chunk_max;
        const Cut c = cut_of(p, args.group, args.prefix, args.D, args.len_q, args.len_k);
        args.pieces = p.kernel == Kernel::near ? p.shares : c.tiles * c.chunks;
    };
    auto run = [&](const AttnArgs& args, const Pass& p) {
        switch (p.kernel) {
            case Kernel::few: return launch_attn_few(args, int(p.grid), s);
            case Kernel::near: return launch_attn_near(args, int(p.grid), s);
            case Kernel::tile: return launch_attn_tile(args, int(p.grid), s);
            default: return launch_attn_wide(args, int(p.grid), s);
        }
    };
    AttnArgs p = a;
    if (P.apart) {
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
        p.part_n = nullptr;
        cut(p, P.prefix);
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
    cut(a, P.own);
    if (P.apart && P.prefix.kernel == Kernel::tile && P.own.kernel == Kernel::few) {
        st = launch_attn_pair(p, int(P.prefix.grid), a, int(P.own.grid), s);
    } else {
        if (P.apart) st = run(p, P.prefix);
        if (st == LYNX_OK) st = run(a, P.own);
    }
    if (st != LYNX_OK) return st;
    if (P.slots > 0) {
        st = launch_attn_join(a, a.slot0, s);
        if (st != LYNX_OK) return st;
    }
    return debug_sync(st, s);
}

}  // extern "C"
