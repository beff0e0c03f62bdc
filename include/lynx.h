/*
 * lynx.h - C ABI of the RT-Lynx sparse + LoRA linear layer for AMD MI355X (gfx950),
 * its dense and 8-bit alternatives, the norms that stand between such layers, and
 * what stands between the QKV and the output projection of a block: rotary positions
 * and attention.
 *
 * The layer (RT-Lynx page, aitrends.kr, "RT-Lynx: Diffusion Transformers에서
 * GEMM Sparsity를 Activation으로 옮겨 실현하는 방법"; section 방법론, item
 * "핵심 메커니즘", and the two formulas of section 코드 예제):
 *
 *     X~   = X with, in every group of 4 consecutive input channels, only the
 *            two entries of largest |x| kept (Top-K 2:4 activation selection)
 *     s    = ||X||_2 / ||X~||_2 per token (row)      (Norm Compensation)
 *     Y    = s * (X~ W^T) + (X LB^T) LA^T           (= S(X) W^T + X (LA LB)^T)
 *
 * Readings fixed by this library where the page is silent:
 *   - groups are 4 consecutive channels of the reduction axis K, aligned at 0
 *     mod 4; ties in |x| go to the lower channel index; -0 and +0 are equal;
 *   - the page's eps is 0; a row whose X~ is zero (only an all-zero row) has s = 1;
 *   - the LoRA branch takes the dense, unscaled X; no bias.
 *
 * Conventions common to every entry point
 *   - bf16 tensors are passed as uint16_t bit patterns.
 *   - Every tensor pointer is a DEVICE pointer owned by the caller; tensors are
 *     contiguous; X, W, LA, LB, T and Y are row-major, the packed operand is
 *     stored as described below; every pointer must be 16-byte aligned.
 *   - Every call is asynchronous on `stream` (a hipStream_t; NULL = default
 *     stream).  The library never allocates device memory, never synchronizes
 *     (outside the debug mode below) and keeps no per-call state, so calls are
 *     re-entrant; concurrent calls that write the same buffers race, as with
 *     any kernel.
 *   - All arguments are validated before anything is launched.  On an error
 *     the status is returned and no output is written.
 *   - Asynchronous device faults surface at the caller's next synchronization
 *     with the stream, not as a status of the call that queued the work.
 *   - Debug mode: with the environment variable LYNX_DEBUG set to anything but
 *     "" or "0" (read on every call), a call that queued work waits for
 *     `stream` before it returns, and a failure of that wait (a fault of this
 *     call's kernels or of earlier work on the stream) is returned as
 *     LYNX_ERR_DEVICE.  A stream that is being captured into a graph is not
 *     waited for.  It serializes the caller; it is meant for debugging.
 *   - Inputs must be finite; NaN/Inf inputs give unspecified outputs.
 *   - Shape limits: K is a positive multiple of 64; M >= 0 and N >= 0 (0 is a
 *     no-op); R (LoRA rank) is one of 0, 16, 32, 48, 64 (0 = no LoRA branch);
 *     M, N, K <= 2^24; (M + 256) * K, (N + 256) * K and (M + 256) * N are each
 *     below 2^31 (every tensor, padded by one 256-row tile, smaller than 2^31
 *     elements, so that 32-bit byte offsets cover it).
 *   - The current device must be gfx950 (MI350 series); otherwise
 *     LYNX_ERR_UNSUPPORTED_DEVICE.
 *
 * Packed sparse operand (the 2:4 activation in the sparse matrix unit's
 * format, which the page has the sparsifier emit directly).  Per row:
 *   values row, K/2 bf16: the two kept entries of every group, in ascending
 *                channel order, copied bit-exactly from X (unscaled);
 *   meta row, K/8 bytes: a 4-bit code per group, (first kept position) |
 *                (second kept position) << 2, positions 0..3 inside the group,
 *                first < second; group 2j in the low nibble of byte j,
 *                group 2j+1 in the high nibble.
 * Storage order: tiles of 16 rows x 64 channels, the A operand of one
 * v_smfmac_f32_16x16x64_bf16 step, each tile contiguous.  With
 * Mp = M rounded up to a multiple of 16:
 *   values [Mp/16][K/64][16][32] bf16  (Mp * K/2 elements): kept value j of
 *          row m at ((m/16)*(K/64) + j/32)*512 + (m%16)*32 + j%32;
 *   meta   [Mp/16][K/64][16][8] uint8  (Mp * K/8 bytes): meta byte j of row m
 *          at ((m/16)*(K/64) + j/8)*128 + (m%16)*8 + j%8.
 * Rows M..Mp-1 are written as zero values and meta 0x44 (positions 0 and 1).
 * The 8 meta bytes of a row and step, read as four little-endian 16-bit
 * words, are the sparse-index operands of the row's four lane groups.
 *   scale  [M] fp32  : s per row;
 *   T      [M][R] bf16 (row-major): X LB^T, the LoRA down-projection of X.
 */
#ifndef LYNX_H
#define LYNX_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void* lynx_stream_t; /* a hipStream_t */

typedef enum lynx_status {
    LYNX_OK = 0,
    LYNX_ERR_NULL = 1,               /* a required pointer is NULL */
    LYNX_ERR_SHAPE = 2,              /* a size is outside the limits above */
    LYNX_ERR_ALIGN = 3,              /* a pointer is not 16-byte aligned */
    LYNX_ERR_WORKSPACE = 4,          /* workspace is NULL or too small */
    LYNX_ERR_DEVICE = 5,             /* a HIP call or a kernel launch failed */
    LYNX_ERR_UNSUPPORTED_DEVICE = 6, /* the current device is not gfx950 */
    LYNX_ERR_SCRATCH = 7             /* the problem does not fit the static scratch array
                                        of lynx_linear_sparse_lora_noalloc */
} lynx_status;

/* Human-readable name of a status; never NULL. */
const char* lynx_status_string(lynx_status s);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int lynx_version(void);

/*
 * Bytes of device workspace lynx_linear_sparse_lora needs for an (M, K, R)
 * problem: the packed operand (values Mp*K bytes, meta Mp*K/8, scale 4M) and
 * T (2MR), each 256-byte aligned.  Returns 0 for invalid sizes.
 */
size_t lynx_workspace_bytes(int64_t M, int64_t K, int64_t R);

/*
 * lynx_sparsify - online activation sparsification and LoRA down-projection.
 * Page: 방법론 "핵심 메커니즘" (Top-K 2:4 selection, S(X) = s X~) and
 * 핵심 기여 (pattern decision, Top-K and compression in one execution path,
 * emitting the sparse-unit layout).  One read of X produces:
 *   values (Mp*K/2 bf16), meta (Mp*K/8 bytes), scale [M] - the packed operand;
 *   T [M][R] = X LB^T (fp32 accumulation, rounded to bf16), if R > 0.
 * Inputs: X [M][K] bf16; LB [R][K] bf16 (NULL iff R == 0); T NULL iff R == 0.
 */
lynx_status lynx_sparsify(const uint16_t* X, const uint16_t* LB,
                          int64_t M, int64_t K, int64_t R,
                          uint16_t* values, uint8_t* meta, float* scale, uint16_t* T,
                          lynx_stream_t stream);

/*
 * lynx_linear_sparse_lora - the whole layer Y = S(X) W^T + X (LA LB)^T.
 * Page: 코드 예제, second formula; 방법론 "CUDA 커널 최적화" (the LoRA output
 * is produced and accumulated on chip inside the sparse GEMM).
 * Runs lynx_sparsify into `workspace`, then the 2:4 sparse-MFMA GEMM whose
 * epilogue adds T LA^T and applies s, with fp32 accumulation and a bf16
 * (round-to-nearest-even) store.
 * Inputs: X [M][K], W [N][K], LA [N][R], LB [R][K] (LA, LB NULL iff R == 0).
 * Output: Y [M][N] bf16.  workspace: >= lynx_workspace_bytes(M, K, R) bytes,
 * 256-byte aligned, contents on entry irrelevant, clobbered.
 */
lynx_status lynx_linear_sparse_lora(const uint16_t* X, const uint16_t* W,
                                    const uint16_t* LA, const uint16_t* LB, uint16_t* Y,
                                    int64_t M, int64_t N, int64_t K, int64_t R,
                                    void* workspace, size_t workspace_bytes,
                                    lynx_stream_t stream);

/*
 * lynx_linear_sparse_lora_noalloc - lynx_linear_sparse_lora without a
 * workspace argument, for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc.  Same inputs, output, kernels and results as
 * lynx_linear_sparse_lora; the packed operand, s and T go to a static device
 * array of the library (64 MiB per device, LYNX_SCRATCH_BYTES), allocated
 * when the library's code is loaded on a device and held until the process
 * ends.  The call itself allocates nothing, on the device or the host.
 *   - Problems whose lynx_workspace_bytes(M, K, R) exceeds LYNX_SCRATCH_BYTES
 *     return LYNX_ERR_SCRATCH (e.g. M = 4096 fits up to K = 12288 with
 *     R = 64; M = 9216 fits up to K = 6144).
 *   - Every call on a device shares that device's array, which keeps the last
 *     call's contents (each call writes every byte it reads before reading
 *     it).  Calls that overlap on one device - on different streams, or from
 *     different host threads without ordering - race on the array and give
 *     undefined results; calls on one stream are ordered and safe.
 *   - The first call on each device looks up the array's device address
 *     (hipGetSymbolAddress) and keeps it; a failure there returns
 *     LYNX_ERR_DEVICE.
 */
#define LYNX_SCRATCH_BYTES ((size_t)64 << 20)

lynx_status lynx_linear_sparse_lora_noalloc(const uint16_t* X, const uint16_t* W,
                                            const uint16_t* LA, const uint16_t* LB, uint16_t* Y,
                                            int64_t M, int64_t N, int64_t K, int64_t R,
                                            lynx_stream_t stream);

/*
 * lynx_linear_sparse_lora_packed - the GEMM half of the layer on an already
 * packed operand: Y = scale * (X~ W^T) + T LA^T, X~ given by values + meta.
 * Same page passages as lynx_linear_sparse_lora.  Used to time the sparse
 * GEMM apart from the sparsifier.  T and LA NULL iff R == 0.
 */
lynx_status lynx_linear_sparse_lora_packed(const uint16_t* values, const uint8_t* meta,
                                           const float* scale, const uint16_t* T,
                                           const uint16_t* W, const uint16_t* LA, uint16_t* Y,
                                           int64_t M, int64_t N, int64_t K, int64_t R,
                                           lynx_stream_t stream);

/*
 * lynx_linear_dense - the dense layer Y = X W^T, bf16 MFMA, fp32 accumulate,
 * bf16 store: the baseline the page's speedups are quoted against
 * (주요 결과, speed/efficiency item).  No LoRA branch.
 */
lynx_status lynx_linear_dense(const uint16_t* X, const uint16_t* W, uint16_t* Y,
                              int64_t M, int64_t N, int64_t K, lynx_stream_t stream);

/*
 * A sequence of linear layers, each either sparse + LoRA or dense: the
 * block-level driver of selective layer skipping (방법론 "핵심 메커니즘",
 * Selective Layer Skipping; 구현 및 학습 세부: in single-stream blocks some
 * layers, e.g. Out/OUp, are left out of the sparsification).  A skipped
 * layer is the original dense layer Y = X W^T (no LoRA branch, which only
 * corrects the sparse one).
 */
typedef enum lynx_layer_mode {
    LYNX_LAYER_SPARSE_LORA = 0,  /* Y = S(X) W^T + X (LA LB)^T, as lynx_linear_sparse_lora */
    LYNX_LAYER_DENSE = 1         /* Y = X W^T, as lynx_linear_dense; LA, LB, R ignored */
} lynx_layer_mode;

typedef struct lynx_layer {
    const uint16_t* X;   /* [M][K] bf16 */
    const uint16_t* W;   /* [N][K] bf16 */
    const uint16_t* LA;  /* [N][R] bf16, NULL iff R == 0 or the layer is dense */
    const uint16_t* LB;  /* [R][K] bf16, NULL iff R == 0 or the layer is dense */
    uint16_t* Y;         /* [M][N] bf16 output */
    int64_t M, N, K, R;
    int32_t mode;        /* a lynx_layer_mode */
} lynx_layer;

/*
 * Bytes of workspace lynx_linear_sequence needs: the largest
 * lynx_workspace_bytes(M, K, R) over its sparse layers (0 if there are none,
 * or if any layer is invalid).  layers: host array of n descriptors.
 */
size_t lynx_sequence_workspace_bytes(const lynx_layer* layers, int64_t n);

/*
 * Runs the n layers in order on `stream` (host array of n descriptors; every
 * pointer inside is a device pointer).  All layers are validated before any
 * launch; on an error nothing is written and the first failing layer's status
 * is returned.  workspace: >= lynx_sequence_workspace_bytes(layers, n) bytes,
 * 256-byte aligned (NULL allowed when no layer is sparse), shared by the
 * sparse layers one after another, contents on entry irrelevant, clobbered.
 * n == 0 is a no-op.  Layers must not write an input of a later layer unless
 * that order is intended: they run exactly in sequence.
 */
lynx_status lynx_linear_sequence(const lynx_layer* layers, int64_t n, void* workspace,
                                 size_t workspace_bytes, lynx_stream_t stream);

/*
 * ---- 8-bit linear layer -----------------------------------------------------
 * Y = Q(X) Q(W)^T with both operands in e4m3 (OCP: 4 exponent bits, 3 fraction
 * bits, largest value 448) and one power-of-two scale per block of 128:
 *   - an activation has a scale for every 128 consecutive channels of a row, a
 *     weight one for every block of 128 rows x 128 channels, both aligned at 0
 *     (where K % 128 == 64 the last block has 64 channels);
 *   - a block whose largest magnitude is a gets the scale 2^e with the smallest
 *     integer e >= -127 that keeps a <= 448 * 2^e (a = 0: e = 0), and the values
 *     x * 2^-e rounded to nearest even.  x * 2^-e is exact, so values and scales
 *     are those of the definition, bit for bit;
 *   - the scale is stored as its E8M0 byte e + 127.  A block that holds a NaN or
 *     an infinity gets the byte 255 (NaN) and unspecified values, and every
 *     output made from it is NaN.  (This path defines them; the rest of the
 *     library leaves non-finite inputs unspecified.)
 * The product takes any operand of this form, also one quantised elsewhere:
 *   Y[m][n] = sum over K blocks kb of 2^(eX[m][kb] + eW[n/128][kb]) *
 *             sum over k in kb of Xq[m][k] Wq[n][k],
 * one rounding to bf16.  The matrix instruction adds products in groups of 8
 * channels, keeping bits down to 2^-13 of the group's largest product, and adds the
 * groups and the accumulator in fp32.
 *
 * Storage: values row-major, Xq [M][K] and Wq [N][K] bytes.
 *   Activation scales [KW][M][4] bytes, KW = ceil(K / 512): the byte of row m and
 *     block kb at ((kb / 4) * M + m) * 4 + kb % 4 (four blocks of a row to a word).
 *   Weight scales [ceil(N / 128)][4 * KW] bytes: block (nb, kb) at nb * 4 * KW + kb.
 *   Places of blocks past K are written as 127 and never used.
 * Shape limits and conventions as above (K a positive multiple of 64).
 */

/* X [M][K] bf16 -> q [M][K], scale [KW][M][4]. */
lynx_status lynx_quantize_fp8(const uint16_t* X, int64_t M, int64_t K, uint8_t* q,
                              uint8_t* scale, lynx_stream_t stream);

/* W [N][K] bf16 -> q [N][K], scale [ceil(N/128)][4 KW]. */
lynx_status lynx_quantize_fp8_weight(const uint16_t* W, int64_t N, int64_t K, uint8_t* q,
                                     uint8_t* scale, lynx_stream_t stream);

/*
 * Bytes of device workspace lynx_linear_fp8 needs for an (M, N, K) layer: the
 * activation's values and scales, each 256-byte aligned; 0 where it needs none (few
 * rows or few output tiles: X is quantised inside the product) and for invalid sizes.
 */
size_t lynx_fp8_workspace_bytes(int64_t M, int64_t N, int64_t K);

/*
 * The whole layer: quantises X (into `workspace`, where it needs one), then the
 * product; on a device of 256 compute units the same Y, bit for bit, as
 * lynx_quantize_fp8 and lynx_linear_fp8_packed (on another, sums may be ordered
 * otherwise).
 * Inputs: X [M][K] bf16; Wq, Ws a quantised weight [N][K].  Output: Y [M][N] bf16.
 * workspace: >= lynx_fp8_workspace_bytes(M, N, K) bytes, 256-byte aligned, contents
 * on entry irrelevant, clobbered; NULL is allowed where that is 0.
 */
lynx_status lynx_linear_fp8(const uint16_t* X, const uint8_t* Wq, const uint8_t* Ws, uint16_t* Y,
                            int64_t M, int64_t N, int64_t K, void* workspace,
                            size_t workspace_bytes, lynx_stream_t stream);

/* The product alone, on a quantised activation Xq, Xs. */
lynx_status lynx_linear_fp8_packed(const uint8_t* Xq, const uint8_t* Xs, const uint8_t* Wq,
                                   const uint8_t* Ws, uint16_t* Y, int64_t M, int64_t N,
                                   int64_t K, lynx_stream_t stream);

/*
 * ---- block norms ------------------------------------------------------------
 * What stands between two linear layers of a transformer block, in one pass:
 *   z  = post(y)                            the norm after the branch
 *   x' = residual_scale * x + gate[b] * z   the residual stream, stored in x_out
 *   h  = pre(x') * (1 + scale[b]) + shift[b]   the next branch's input
 * post and pre are each one of
 *   LYNX_NORM_NONE    post: z = y.  pre: no h (h, q and pre's parameters NULL);
 *   LYNX_NORM_RMS     v / sqrt(mean(v^2) + eps) * weight + bias;
 *   LYNX_NORM_LAYER   (v - mean(v)) / sqrt(var(v) + eps) * weight + bias;
 * over the C channels of a row, with an absent (NULL) weight, scale or gate read
 * as no factor and an absent bias or shift as no term.  Rows are samples of
 * M / samples rows each, b the row's sample.  All arithmetic is fp32, and h is
 * taken from x' before x' is rounded for x_out.  A channel's given parameters are
 * combined first, into one factor and one term: weight * (1 + scale) and
 * bias * (1 + scale) + shift, post_weight * gate and post_bias * gate.  So where one
 * of them is infinite, a given bias of the other sign (or 0) makes NaN.
 *   - y == NULL: no branch; x' = x, and x_out, gate, post_weight and post_bias are
 *     NULL and residual_scale is not used.
 *   - h is written as bf16 to `h`, or as the 8-bit operand (quantised from the
 *     fp32 h; C % 64 == 0) to `q` [M][C] and `q_scale`: exactly one form is given
 *     when pre is not LYNX_NORM_NONE.
 *   - x and x_out are bf16, or fp32 where x_fp32 is not 0.  x_out may be x; no
 *     other output may overlap an input.
 *   - A norm makes a row NaN throughout (h, with every scale of the 8-bit form; after
 *     a post norm x' too) where the row it is taken of holds a NaN or an infinity, or
 *     values so large that a sum of them or of their squares passes fp32's range (one of
 *     2e19 does, or many smaller ones).  Where y has no post norm, a NaN or an infinity in
 *     x or y makes x' so in its channel alone.  No other row changes.
 * Limits: C a multiple of 8, 8 <= C <= 16384; 0 <= M <= 2^23 (0 is a no-op);
 * samples >= 1 divides M; strides (in elements, from one sample's row to the
 * next; 0 = one row for all) >= 0 and multiples of 8; eps and post_eps >= 0.
 * Every pointer is 16-byte aligned.
 */
typedef enum lynx_norm_kind {
    LYNX_NORM_NONE = 0,
    LYNX_NORM_RMS = 1,
    LYNX_NORM_LAYER = 2
} lynx_norm_kind;

typedef struct lynx_norm {
    const void* x;                /* [M][C] bf16 or fp32 */
    const uint16_t* y;            /* [M][C] bf16, or NULL */
    const uint16_t* gate;         /* samples rows of C bf16, gate_stride apart, or NULL */
    const uint16_t* post_weight;  /* [C] bf16 or NULL; NULL if post_norm is NONE */
    const uint16_t* post_bias;    /* [C] bf16 or NULL; NULL if post_norm is NONE */
    const uint16_t* weight;       /* [C] bf16 or NULL */
    const uint16_t* bias;         /* [C] bf16 or NULL */
    const uint16_t* scale;        /* samples rows, scale_stride apart, or NULL */
    const uint16_t* shift;        /* samples rows, shift_stride apart, or NULL */
    void* x_out;                  /* [M][C] as x; NULL iff y is NULL */
    uint16_t* h;                  /* [M][C] bf16, or NULL */
    uint8_t* q;                   /* [M][C] e4m3, or NULL */
    uint8_t* q_scale;             /* [ceil(C/512)][M][4], NULL iff q is NULL */
    int64_t M, C, samples;
    int64_t gate_stride, scale_stride, shift_stride;
    float residual_scale, post_eps, eps;
    int32_t x_fp32;
    int32_t post_norm, norm;      /* lynx_norm_kind */
} lynx_norm;

lynx_status lynx_block_norm(const lynx_norm* norm, lynx_stream_t stream);

/*
 * ---- rotary positions -------------------------------------------------------
 * q and k between their projection and attention, in one pass: the optional rms norm
 * of each head, then a turn of pairs of channels by the token's positions on up to
 * four axes (time, height, width, ...):
 *   x <- x / sqrt(mean(x^2) + eps) * weight      norm LYNX_NORM_RMS, over the D
 *                                                channels of a head; weight NULL: 1
 *   (x_m, x_n) <- (x_m cos a - x_n sin a, x_m sin a + x_n cos a)
 * Axis i turns axis_dims[i] channels; R is their sum.  The R / 2 pairs go to the axes
 * in order; pair p, the j-th of its axis i, turns by
 *   a = positions[t][i] * theta^(-2 j / axis_dims[i])   LYNX_LADDER_AXIS: every axis
 *                                                       has frequencies of its own;
 *   a = positions[t][i] * theta^(-2 p / R)              LYNX_LADDER_JOINT: the axes
 *                                                       share one row of frequencies.
 * Pair p is channels 2 p and 2 p + 1 (LYNX_PAIRS_ADJACENT), or p and p + R / 2
 * (LYNX_PAIRS_HALVES).  Channels from R on are normed but not turned.
 * Angles are taken in 64 bits, off by 2^-52 of themselves at most, and reduced to one turn
 * before they are rounded to fp32 (2^-26 of a turn): an angle of 2^31 is within 2^-23 of a
 * turn.  Norm and turn are fp32, and there is one rounding to bf16.
 *   - The turn is undone (the backward pass of a turn without a norm) by the same call
 *     with negated positions.
 *   - Strides are in elements, between tokens and between heads, multiples of 8, and
 *     not negative; channels are contiguous.  So q and k may be slices of one
 *     projection's output.
 *   - q_out may be q and k_out k, with the same strides; else no output may overlap an
 *     input, and no two rows of outputs may overlap.
 *   - A head whose row holds a NaN or an infinity, or whose squares pass fp32's range,
 *     becomes NaN throughout under a norm.  Without one, NaN and infinities reach their
 *     pair alone.  A position that is not finite makes its axis' pairs NaN.
 *   - Squares below 2^-126 lose bits, and below 2^-149 all of them: with eps 0 a row whose
 *     channels are all below 2^-63 is inexact, infinite or NaN under a norm.
 * Limits: head_dim a multiple of 8, 8..256; 1 to 4 axes, each of an even number >= 2
 * of channels, R <= head_dim; theta normal and > 0; 0 <= tokens <= 2^24 (0 is a no-op);
 * 1 <= q_heads, 0 <= k_heads (0: k, k_out and k_weight are NULL), each <= 1024; tokens *
 * (q_heads + k_heads) < 2^31; eps >= 0.  Pointers are 16-byte aligned.
 */
typedef enum lynx_pairs { LYNX_PAIRS_ADJACENT = 0, LYNX_PAIRS_HALVES = 1 } lynx_pairs;
typedef enum lynx_ladder { LYNX_LADDER_AXIS = 0, LYNX_LADDER_JOINT = 1 } lynx_ladder;

typedef struct lynx_rotary {
    const uint16_t* q;        /* tokens x q_heads rows of head_dim bf16 */
    const uint16_t* k;        /* tokens x k_heads rows, or NULL */
    const uint16_t* q_weight; /* [head_dim] bf16 or NULL; NULL if norm is NONE */
    const uint16_t* k_weight; /* [head_dim] bf16 or NULL; NULL if norm is NONE */
    const void* positions;    /* [tokens][axes] int32, or fp32 */
    uint16_t* q_out;
    uint16_t* k_out;
    int64_t tokens, q_heads, k_heads, head_dim;
    int64_t q_stride, q_head_stride, k_stride, k_head_stride;
    int64_t q_out_stride, q_out_head_stride, k_out_stride, k_out_head_stride;
    double theta;
    int32_t axis_dims[4];     /* places from `axes` on are not read */
    int32_t axes;
    int32_t positions_fp32;   /* 0: int32 */
    int32_t pairs, ladder;    /* lynx_pairs, lynx_ladder */
    int32_t norm;             /* LYNX_NORM_NONE or LYNX_NORM_RMS */
    float eps;
} lynx_rotary;

lynx_status lynx_qk_rotary(const lynx_rotary* rotary, lynx_stream_t stream);

/*
 * ---- attention --------------------------------------------------------------
 * For every query row (token and head) over the keys that it sees:
 *   out = sum_j p_j v_j / sum_j p_j,   p_j = exp(scale * q . k_j)
 *   lse = log(sum_j p_j)               natural logarithm, fp32, if lse is given
 * q has `heads` heads, k and v `kv_heads`; head h reads key head h / (heads / kv_heads).
 * A call works on `batch` sequences, given in one of two ways:
 *   packed   cu_q, cu_k (device, batch + 1 int32 each): sequence s has the query tokens
 *            cu_q[s] .. cu_q[s+1] - 1 and the key tokens cu_k[s] .. cu_k[s+1] - 1, any
 *            number of either, also none.  The *_batch_stride are not used.
 *   uniform  cu_q and cu_k NULL: every sequence has tokens_q / batch query tokens and
 *            tokens_k / batch key tokens, sequences *_batch_stride apart.
 * A sequence's query i of Lq sees all of its Lk keys or, with `causal`, the keys
 * j <= i + Lk - Lq (the last query sees every key: single tokens on a cache that
 * already holds their own keys).  With a prefix (prefix_tokens > 0), every query of every
 * sequence also sees all prefix keys, which come before the sequence's own; causal
 * concerns own keys alone.  A query that sees no key gets out = 0 and lse = -infinity.
 *   - Scores, times scale too, and sums are fp32.  p_j, taken relative to a power of two no
 *     further than 2^9 below the row's largest (2^25 for scores past 2^23), is rounded to
 *     bf16, for its product with v_j and for out's divisor alike (lse sums the p_j before
 *     that); out has one more rounding.  out's sums round once for every 16 keys (n / 16 2^-24
 *     relative at most), lse's sum keeps what its additions lose.  A row's result does not
 *     depend on what other rows hold, and is the same in every call of the same sizes, offsets
 *     and strides.
 *   - Keys that a query does not see have no influence on it, whatever they hold; with
 *     NaN or infinities among the keys and values that it sees, its row is as the
 *     formula gives it (an infinite or NaN value whose p_j is 0 makes NaN), and so with a
 *     score that passes fp32's range; but scores that are all -infinity count as no key seen.
 *   - Rows of out and lse before cu_q[0] and from cu_q[batch] on are left as they were.
 *     Offsets must not decrease and lie within 0 .. tokens_q (tokens_k); the device checks
 *     this only so far that no memory beside the tensors is touched: results of other offsets
 *     are unspecified.
 *   - Strides are in elements, multiples of 8, not negative; channels are contiguous.
 *     Token strides of k, v and the prefix are at least head_dim and below 2^23.  Heads
 *     may share memory (head stride 0) in inputs.  out overlaps no input, and its rows
 *     do not overlap.
 *   - Sequences of any length may be mixed.  Which kernel runs, and whether keys are
 *     split over workgroups and joined, follows from the totals, so calls whose sequences
 *     are alike in length are the fastest.
 * Limits: head_dim a multiple of 8, 8..128; 1 <= kv_heads, heads a multiple of it, <= 1024;
 * 1 <= batch <= 2^16; tokens_q, tokens_k and prefix_tokens each 0..2^26 (tokens_q == 0
 * is a no-op), in the uniform form multiples of batch; tokens_q * heads < 2^30; batch *
 * kv_heads <= 2^21; 0 < scale < 2^127.  q, k, v, out and prefix pointers are 16-byte
 * aligned, cu_* and lse 4-byte.  k and v may be NULL if tokens_k is 0.
 */
typedef struct lynx_attn {
    const uint16_t* q;        /* bf16 */
    const uint16_t* k;
    const uint16_t* v;
    const uint16_t* prefix_k; /* prefix_tokens x kv_heads rows of head_dim, or NULL */
    const uint16_t* prefix_v;
    const int32_t* cu_q;      /* both, or neither */
    const int32_t* cu_k;
    uint16_t* out;            /* tokens_q x heads rows of head_dim */
    float* lse;               /* [tokens_q][heads], or NULL */
    int64_t batch, tokens_q, tokens_k, prefix_tokens;
    int64_t heads, kv_heads, head_dim;
    int64_t q_batch_stride, q_stride, q_head_stride;
    int64_t k_batch_stride, k_stride, k_head_stride;
    int64_t v_batch_stride, v_stride, v_head_stride;
    int64_t out_batch_stride, out_stride, out_head_stride;
    int64_t prefix_k_stride, prefix_k_head_stride, prefix_v_stride, prefix_v_head_stride;
    float scale;
    int32_t causal;
} lynx_attn;

/*
 * Bytes of device workspace lynx_attention needs for these sizes, causal or not, and
 * offsets given (cu_q not NULL) or not; nothing else is looked at.  0 where it needs none, and
 * for invalid sizes.  Contents on entry irrelevant, clobbered; 256-byte aligned; NULL is
 * allowed where it is 0.  Calls that may overlap need workspaces of their own.
 */
size_t lynx_attention_workspace_bytes(const lynx_attn* attn);

lynx_status lynx_attention(const lynx_attn* attn, void* workspace, size_t workspace_bytes,
                           lynx_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LYNX_H */
