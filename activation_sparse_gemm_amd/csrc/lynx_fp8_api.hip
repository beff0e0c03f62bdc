// C ABI of the 8-bit linear layer and of the block norms: argument validation,
// workspace layout and dispatch.  Defined in lynx.h.
#include <initializer_list>

#include "lynx_debug.h"
#include "lynx_fp8.h"

namespace lynx {
namespace {

struct Fp8Layout {
    size_t q, scale, total;
};

Fp8Layout fp8_layout(int64_t M, int64_t N, int64_t K) {
    Fp8Layout L = {0, 0, 0};
    if (fp8_fuse(M, N, K) != Fp8Fuse::no) return L;
    L.q = 0;
    L.scale = round_up256(size_t(M) * size_t(K));
    L.total = L.scale + round_up256(size_t(fp8_scale_words(int(K))) * size_t(M) * 4);
    return L;
}

bool all16(std::initializer_list<const void*> ps) {
    for (const void* p : ps)
        if (!aligned16(p)) return false;
    return true;
}

constexpr int64_t kMaxNormRows = int64_t(1) << 23;
constexpr int64_t kMaxNormC = 16384;  // 8 waves of 4 x 8 channels a lane

bool kind_ok(int32_t k) {
    return k == LYNX_NORM_NONE || k == LYNX_NORM_RMS || k == LYNX_NORM_LAYER;
}

lynx_status validate_norm(const lynx_norm& d, bool* noop) {
    *noop = false;
    if (d.M < 0 || d.M > kMaxNormRows || d.C < 8 || d.C > kMaxNormC || d.C % 8 != 0)
        return LYNX_ERR_SHAPE;
    if (d.samples < 1 || d.M % d.samples != 0) return LYNX_ERR_SHAPE;
    for (int64_t s : {d.gate_stride, d.scale_stride, d.shift_stride})
        if (s < 0 || s % 8 != 0) return LYNX_ERR_SHAPE;
    if (!kind_ok(d.norm) || !kind_ok(d.post_norm)) return LYNX_ERR_SHAPE;
    if (!(d.eps >= 0.f) || !(d.post_eps >= 0.f)) return LYNX_ERR_SHAPE;
    if (d.q && d.C % 64 != 0) return LYNX_ERR_SHAPE;
    if (d.M == 0) {
        *noop = true;
        return LYNX_OK;
    }
    // pointers that have to be there, and pointers that may not
    if (!d.x) return LYNX_ERR_NULL;
    if (d.norm == LYNX_NORM_NONE) {
        if (d.h || d.q || d.q_scale || d.weight || d.bias || d.scale || d.shift)
            return LYNX_ERR_NULL;
        if (!d.y) return LYNX_ERR_NULL;  // nothing to compute
    } else if ((d.h != nullptr) == (d.q != nullptr) || (d.q != nullptr) != (d.q_scale != nullptr)) {
        return LYNX_ERR_NULL;
    }
    if ((d.y != nullptr) != (d.x_out != nullptr)) return LYNX_ERR_NULL;
    if (!d.y && (d.gate || d.post_norm != LYNX_NORM_NONE)) return LYNX_ERR_NULL;
    if (d.post_norm == LYNX_NORM_NONE && (d.post_weight || d.post_bias)) return LYNX_ERR_NULL;
    if (!all16({d.x, d.y, d.gate, d.post_weight, d.post_bias, d.weight, d.bias, d.scale, d.shift,
                d.x_out, d.h, d.q, d.q_scale}))
        return LYNX_ERR_ALIGN;
    return LYNX_OK;
}

}  // namespace
}  // namespace lynx

using namespace lynx;

extern "C" {

lynx_status lynx_quantize_fp8(const uint16_t* X, int64_t M, int64_t K, uint8_t* q, uint8_t* scale,
                              lynx_stream_t stream) {
    if (!dims_ok(M, 1, K)) return LYNX_ERR_SHAPE;
    if (M == 0) return LYNX_OK;
    if (!X || !q || !scale) return LYNX_ERR_NULL;
    if (!all16({X, q, scale})) return LYNX_ERR_ALIGN;
    const lynx_status st = check_device();
    if (st != LYNX_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return debug_sync(launch_quantize_fp8(X, int(M), int(K), q, scale, s), s);
}

lynx_status lynx_quantize_fp8_weight(const uint16_t* W, int64_t N, int64_t K, uint8_t* q,
                                     uint8_t* scale, lynx_stream_t stream) {
    if (!dims_ok(1, N, K)) return LYNX_ERR_SHAPE;
    if (N == 0) return LYNX_OK;
    if (!W || !q || !scale) return LYNX_ERR_NULL;
    if (!all16({W, q, scale})) return LYNX_ERR_ALIGN;
    const lynx_status st = check_device();
    if (st != LYNX_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return debug_sync(launch_quantize_fp8_weight(W, int(N), int(K), q, scale, s), s);
}

size_t lynx_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K) {
    if (!dims_ok(M, N, K)) return 0;
    return fp8_layout(M, N, K).total;
}

lynx_status lynx_linear_fp8(const uint16_t* X, const uint8_t* Wq, const uint8_t* Ws, uint16_t* Y,
                            int64_t M, int64_t N, int64_t K, void* workspace,
                            size_t workspace_bytes, lynx_stream_t stream) {
    if (!dims_ok(M, N, K)) return LYNX_ERR_SHAPE;
    if (M == 0 || N == 0) return LYNX_OK;
    if (!X || !Wq || !Ws || !Y) return LYNX_ERR_NULL;
    if (!all16({X, Wq, Ws, Y})) return LYNX_ERR_ALIGN;
    const Fp8Layout L = fp8_layout(M, N, K);
    if (L.total > 0) {
        if (!workspace || workspace_bytes < L.total) return LYNX_ERR_WORKSPACE;
        if ((reinterpret_cast<uintptr_t>(workspace) & 255u) != 0) return LYNX_ERR_ALIGN;
    }
    lynx_status st = check_device();
    if (st != LYNX_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    const Fp8Fuse fuse = fp8_fuse(M, N, K);
    if (fuse == Fp8Fuse::few)
        return debug_sync(launch_gemm_fp8_few(X, nullptr, Wq, Ws, Y, int(M), int(N), int(K), s), s);
    if (fuse != Fp8Fuse::no)
        return debug_sync(
            launch_gemm_fp8_mid_quant(X, Wq, Ws, Y, int(M), int(N), int(K), fuse, s), s);
    uint8_t* q = static_cast<uint8_t*>(workspace) + L.q;
    uint8_t* scale = static_cast<uint8_t*>(workspace) + L.scale;
    st = launch_quantize_fp8(X, int(M), int(K), q, scale, s);
    if (st != LYNX_OK) return st;
    return debug_sync(launch_gemm_fp8(q, scale, Wq, Ws, Y, int(M), int(N), int(K), s), s);
}

lynx_status lynx_linear_fp8_packed(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                                   const uint8_t* Ws, uint16_t* Y, int64_t M, int64_t N, int64_t K,
                                   lynx_stream_t stream) {
    if (!dims_ok(M, N, K)) return LYNX_ERR_SHAPE;
    if (M == 0 || N == 0) return LYNX_OK;
    if (!Xq || !Xs || !Wq || !Ws || !Y) return LYNX_ERR_NULL;
    if (!all16({Xq, Xs, Wq, Ws, Y})) return LYNX_ERR_ALIGN;
    const lynx_status st = check_device();
    if (st != LYNX_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return debug_sync(launch_gemm_fp8(Xq, Xs, Wq, Ws, Y, int(M), int(N), int(K), s), s);
}

lynx_status lynx_block_norm(const lynx_norm* norm, lynx_stream_t stream) {
    if (!norm) return LYNX_ERR_NULL;
    const lynx_norm d = *norm;
    bool noop = false;
    lynx_status st = validate_norm(d, &noop);
    if (st != LYNX_OK || noop) return st;
    st = check_device();
    if (st != LYNX_OK) return st;
    const hipStream_t s = static_cast<hipStream_t>(stream);
    return debug_sync(launch_block_norm(d, s), s);
}

}  // extern "C"
