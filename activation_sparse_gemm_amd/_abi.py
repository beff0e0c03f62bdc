"""ctypes binding of liblynx.so (include/lynx.h, include/lynx_probe.h).

Argument marshalling only: tensors are checked for device, dtype, shape and
contiguity, then their data pointers and torch's current HIP stream are passed
to the C entry points.  Every computation runs in the library's HIP kernels;
there is no fallback.  If the library is not built, every call raises.
"""
from __future__ import annotations

import ctypes
import os
import struct

import torch

_PKG = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_PKG, "liblynx.so")

LYNX_OK = 0
STATUS_NAMES = {
    0: "LYNX_OK", 1: "LYNX_ERR_NULL", 2: "LYNX_ERR_SHAPE", 3: "LYNX_ERR_ALIGN",
    4: "LYNX_ERR_WORKSPACE", 5: "LYNX_ERR_DEVICE", 6: "LYNX_ERR_UNSUPPORTED_DEVICE",
    7: "LYNX_ERR_SCRATCH",
}
SCRATCH_BYTES = 64 << 20  # LYNX_SCRATCH_BYTES

LAYER_SPARSE_LORA, LAYER_DENSE = 0, 1


class Layer(ctypes.Structure):
    """struct lynx_layer (include/lynx.h)."""
    _fields_ = [("X", ctypes.c_void_p), ("W", ctypes.c_void_p), ("LA", ctypes.c_void_p),
                ("LB", ctypes.c_void_p), ("Y", ctypes.c_void_p), ("M", ctypes.c_int64),
                ("N", ctypes.c_int64), ("K", ctypes.c_int64), ("R", ctypes.c_int64),
                ("mode", ctypes.c_int32)]


NORM_KINDS = {None: 0, "rms": 1, "layer": 2}


class Norm(ctypes.Structure):
    """struct lynx_norm (include/lynx.h)."""
    _fields_ = ([(n, ctypes.c_void_p) for n in
                 ("x", "y", "gate", "post_weight", "post_bias", "weight", "bias", "scale", "shift",
                  "x_out", "h", "q", "q_scale")]
                + [(n, ctypes.c_int64) for n in ("M", "C", "samples", "gate_stride",
                                                 "scale_stride", "shift_stride")]
                + [(n, ctypes.c_float) for n in ("residual_scale", "post_eps", "eps")]
                + [(n, ctypes.c_int32) for n in ("x_fp32", "post_norm", "norm")])


# the same as bytes: packing it takes a quarter of the time of filling a Structure
_NORM = struct.Struct("@13P6q3f3i")
assert _NORM.size == ctypes.sizeof(Norm)


# every symbol the public headers declare, with (restype, argtypes)
_P, _I64, _I, _SZ = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_size_t
_LP = ctypes.POINTER(Layer)
SIGNATURES = {
    "lynx_status_string": (ctypes.c_char_p, [_I]),
    "lynx_version": (_I, []),
    "lynx_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "lynx_sparsify": (_I, [_P, _P, _I64, _I64, _I64, _P, _P, _P, _P, _P]),
    "lynx_linear_sparse_lora": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P, _SZ, _P]),
    "lynx_linear_sparse_lora_packed": (_I, [_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64,
                                            _P]),
    "lynx_linear_sparse_lora_noalloc": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _P]),
    "lynx_linear_dense": (_I, [_P, _P, _P, _I64, _I64, _I64, _P]),
    "lynx_sequence_workspace_bytes": (_SZ, [_LP, _I64]),
    "lynx_linear_sequence": (_I, [_LP, _I64, _P, _SZ, _P]),
    "lynx_quantize_fp8": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "lynx_quantize_fp8_weight": (_I, [_P, _I64, _I64, _P, _P, _P]),
    "lynx_fp8_workspace_bytes": (_SZ, [_I64, _I64, _I64]),
    "lynx_linear_fp8": (_I, [_P, _P, _P, _P, _I64, _I64, _I64, _P, _SZ, _P]),
    "lynx_linear_fp8_packed": (_I, [_P, _P, _P, _P, _P, _I64, _I64, _I64, _P]),
    "lynx_block_norm": (_I, [_P, _P]),
    "lynx_probe_mfma": (_I, [_I, _I, _P, _P, _P, _P, _P]),
    "lynx_probe_mfma_rate": (_I, [_I, _I, _I, _P, _P, _P]),
}


class LynxError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {status_string(status)}")


_lib = None


def lib() -> ctypes.CDLL:
    """The loaded library; raises if it has not been built."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with `python -m activation_sparse_gemm_amd.build`")
        L = ctypes.CDLL(LIB_PATH)
        for name, (res, args) in SIGNATURES.items():
            fn = getattr(L, name)
            fn.restype = res
            fn.argtypes = args
        _lib = L
    return _lib


def status_string(status: int) -> str:
    return lib().lynx_status_string(int(status)).decode()


def _check(status: int, where: str) -> None:
    if status != LYNX_OK:
        raise LynxError(status, where)


def _ptr(t: torch.Tensor | None) -> int | None:
    return None if t is None else t.data_ptr()


def _stream(device: torch.device) -> int:
    return torch.cuda.current_stream(device).cuda_stream


def _need(t: torch.Tensor, dtype: torch.dtype, shape: tuple, name: str) -> None:
    if t.dtype != dtype:
        raise TypeError(f"{name}: expected {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name}: expected shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name}: must be contiguous")
    if t.device.type != "cuda":
        raise ValueError(f"{name}: must be a device tensor")


def version() -> int:
    return lib().lynx_version()


def workspace_bytes(M: int, K: int, R: int) -> int:
    return lib().lynx_workspace_bytes(M, K, R)


def padded_rows(M: int) -> int:
    """Rows of the stored packed operand: whole 16-row tiles."""
    return (M + 15) // 16 * 16


def sparsify(X: torch.Tensor, LB: torch.Tensor | None = None, out: dict | None = None):
    """Packed 2:4 operand and LoRA down-projection of X (lynx_sparsify).

    Returns (values, meta, scale, T): values (Mp*K/2,) bf16 and meta (Mp*K/8,)
    uint8 in the 16-row x 64-channel tile order of lynx.h (Mp = M rounded up
    to 16), scale [M] fp32, T [M, R] bf16 or None.
    """
    M, K = X.shape
    Mp = padded_rows(M)
    R = 0 if LB is None else LB.shape[0]
    _need(X, torch.bfloat16, (M, K), "X")
    if LB is not None:
        _need(LB, torch.bfloat16, (R, K), "LB")
    dev = X.device
    out = out or {}
    values = out.get("values")
    if values is None:
        values = torch.empty((Mp * K // 2,), dtype=torch.bfloat16, device=dev)
    meta = out.get("meta")
    if meta is None:
        meta = torch.empty((Mp * K // 8,), dtype=torch.uint8, device=dev)
    scale = out.get("scale")
    if scale is None:
        scale = torch.empty((M,), dtype=torch.float32, device=dev)
    T = out.get("T")
    if T is None and R > 0:
        T = torch.empty((M, R), dtype=torch.bfloat16, device=dev)
    _need(values, torch.bfloat16, (Mp * K // 2,), "values")
    _need(meta, torch.uint8, (Mp * K // 8,), "meta")
    _need(scale, torch.float32, (M,), "scale")
    if R > 0:
        _need(T, torch.bfloat16, (M, R), "T")
    _check(lib().lynx_sparsify(_ptr(X), _ptr(LB), M, K, R, _ptr(values), _ptr(meta),
                               _ptr(scale), _ptr(T) if R > 0 else None, _stream(dev)),
           "lynx_sparsify")
    return values, meta, scale, (T if R > 0 else None)


def linear_sparse_lora(X, W, LA=None, LB=None, Y=None, workspace=None):
    """Y = S(X) W^T + X (LA LB)^T (lynx_linear_sparse_lora)."""
    M, K = X.shape
    N = W.shape[0]
    R = 0 if LA is None else LA.shape[1]
    _need(X, torch.bfloat16, (M, K), "X")
    _need(W, torch.bfloat16, (N, K), "W")
    if R > 0:
        _need(LA, torch.bfloat16, (N, R), "LA")
        _need(LB, torch.bfloat16, (R, K), "LB")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _need(Y, torch.bfloat16, (M, N), "Y")
    nbytes = workspace_bytes(M, K, R)
    if workspace is None:
        workspace = torch.empty((max(nbytes, 1),), dtype=torch.uint8, device=X.device)
    _check(lib().lynx_linear_sparse_lora(_ptr(X), _ptr(W), _ptr(LA), _ptr(LB), _ptr(Y), M, N, K,
                                         R, _ptr(workspace), workspace.numel(),
                                         _stream(X.device)),
           "lynx_linear_sparse_lora")
    return Y


def linear_sparse_lora_noalloc(X, W, LA=None, LB=None, Y=None):
    """Y = S(X) W^T + X (LA LB)^T with the library's static scratch array as
    workspace (lynx_linear_sparse_lora_noalloc): the C call allocates nothing.
    Pass Y to keep this wrapper from allocating it."""
    M, K = X.shape
    N = W.shape[0]
    R = 0 if LA is None else LA.shape[1]
    _need(X, torch.bfloat16, (M, K), "X")
    _need(W, torch.bfloat16, (N, K), "W")
    if R > 0:
        _need(LA, torch.bfloat16, (N, R), "LA")
        _need(LB, torch.bfloat16, (R, K), "LB")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _need(Y, torch.bfloat16, (M, N), "Y")
    _check(lib().lynx_linear_sparse_lora_noalloc(_ptr(X), _ptr(W), _ptr(LA), _ptr(LB), _ptr(Y),
                                                 M, N, K, R, _stream(X.device)),
           "lynx_linear_sparse_lora_noalloc")
    return Y


def linear_sparse_lora_packed(values, meta, scale, T, W, LA=None, Y=None):
    """Y = scale * (X~ W^T) + T LA^T from a packed operand (lynx_linear_sparse_lora_packed)."""
    M = scale.shape[0]
    N, K = W.shape
    Mp = padded_rows(M)
    R = 0 if LA is None else LA.shape[1]
    _need(values, torch.bfloat16, (Mp * K // 2,), "values")
    _need(meta, torch.uint8, (Mp * K // 8,), "meta")
    _need(scale, torch.float32, (M,), "scale")
    _need(W, torch.bfloat16, (N, K), "W")
    if R > 0:
        _need(T, torch.bfloat16, (M, R), "T")
        _need(LA, torch.bfloat16, (N, R), "LA")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=W.device)
    _need(Y, torch.bfloat16, (M, N), "Y")
    _check(lib().lynx_linear_sparse_lora_packed(_ptr(values), _ptr(meta), _ptr(scale),
                                                _ptr(T) if R > 0 else None, _ptr(W),
                                                _ptr(LA) if R > 0 else None, _ptr(Y), M, N, K, R,
                                                _stream(W.device)),
           "lynx_linear_sparse_lora_packed")
    return Y


def linear_dense(X, W, Y=None):
    """Y = X W^T (lynx_linear_dense)."""
    M, K = X.shape
    N = W.shape[0]
    _need(X, torch.bfloat16, (M, K), "X")
    _need(W, torch.bfloat16, (N, K), "W")
    if Y is None:
        Y = torch.empty((M, N), dtype=torch.bfloat16, device=X.device)
    _need(Y, torch.bfloat16, (M, N), "Y")
    _check(lib().lynx_linear_dense(_ptr(X), _ptr(W), _ptr(Y), M, N, K, _stream(X.device)),
           "lynx_linear_dense")
    return Y


def _layer_struct(d: dict) -> Layer:
    X, W, Y = d["X"], d["W"], d["Y"]
    M, K = X.shape
    N = W.shape[0]
    dense = d.get("dense", False)
    LA, LB = (None, None) if dense else (d.get("LA"), d.get("LB"))
    R = 0 if LA is None else LA.shape[1]
    _need(X, torch.bfloat16, (M, K), "X")
    _need(W, torch.bfloat16, (N, K), "W")
    _need(Y, torch.bfloat16, (M, N), "Y")
    if R > 0:
        _need(LA, torch.bfloat16, (N, R), "LA")
        _need(LB, torch.bfloat16, (R, K), "LB")
    return Layer(_ptr(X), _ptr(W), _ptr(LA), _ptr(LB), _ptr(Y), M, N, K, R,
                 LAYER_DENSE if dense else LAYER_SPARSE_LORA)


def sequence_workspace_bytes(layers: list) -> int:
    arr = (Layer * len(layers))(*[_layer_struct(d) for d in layers])
    return lib().lynx_sequence_workspace_bytes(arr, len(layers))


def linear_sequence(layers: list, workspace=None):
    """Runs the layers in order (lynx_linear_sequence).  Each layer is a dict
    with X, W, Y (device tensors), LA and LB for a sparse + LoRA layer, and
    dense=True for a skipped (dense) layer."""
    if not layers:
        return
    arr = (Layer * len(layers))(*[_layer_struct(d) for d in layers])
    dev = layers[0]["X"].device
    nbytes = lib().lynx_sequence_workspace_bytes(arr, len(layers))
    if workspace is None and nbytes > 0:
        workspace = torch.empty((nbytes,), dtype=torch.uint8, device=dev)
    _check(lib().lynx_linear_sequence(arr, len(layers), _ptr(workspace),
                                      0 if workspace is None else workspace.numel(),
                                      _stream(dev)),
           "lynx_linear_sequence")


# ---- 8-bit linear layer and block norms ---------------------------------------

FP8, E8M0 = torch.float8_e4m3fn, torch.float8_e8m0fnu


def _expect(t, dtype, shape, dev, name) -> int:
    """The data pointer of a contiguous device tensor of this type and shape on
    `dev`; raises as _need does."""
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous() or t.device != dev:
        _need(t, dtype, shape, name)
        raise ValueError(f"{name}: expected a tensor on {dev}, got one on {t.device}")
    return t.data_ptr()


def _rows(t, dtype, name):
    """(rows, columns, device, data pointer) of a contiguous matrix on a device."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name}: expected a matrix, got shape {tuple(shape)}")
    if not t.is_cuda:
        raise ValueError(f"{name}: must be a device tensor")
    if t.dtype is not dtype or not t.is_contiguous():
        _need(t, dtype, shape, name)
    return shape[0], shape[1], t.device, t.data_ptr()


_fns: dict = {}


def _call(fn: str, dev: torch.device, *args) -> None:
    """Calls the entry point on `dev`'s current stream, with `dev` as the
    current device (the library works on the current device).  Short calls are
    bound by this code's time: the stream handle comes without a Stream object
    around it (0.1 us instead of 2)."""
    f = _fns.get(fn)
    if f is None:
        f = _fns[fn] = getattr(lib(), fn)
    i = dev.index
    if i == torch._C._cuda_getDevice():
        st = f(*args, torch._C._cuda_getCurrentRawStream(i))
    else:
        with torch.cuda.device(dev):
            st = f(*args, torch._C._cuda_getCurrentRawStream(i))
    if st != LYNX_OK:
        raise LynxError(st, fn)


def _scale_words(K: int) -> int:
    return (K + 511) // 512


def quantize_fp8(X: torch.Tensor, out: tuple | None = None):
    """The 8-bit operand of an activation (lynx_quantize_fp8).

    Returns (q, scale): q [M, K] float8_e4m3fn and scale [ceil(K/512), M, 4]
    float8_e8m0fnu, the scale of row m and channels 128 kb .. 128 kb + 127 at
    scale[kb // 4, m, kb % 4].  out: the pair of tensors to write.
    """
    M, K, dev, x = _rows(X, torch.bfloat16, "X")
    words = _scale_words(K)
    if out is None:
        q = torch.empty(M, K, dtype=FP8, device=dev)
        scale = torch.empty(words, M, 4, dtype=E8M0, device=dev)
    else:
        q, scale = out
        _expect(q, FP8, (M, K), dev, "q")
        _expect(scale, E8M0, (words, M, 4), dev, "scale")
    _call("lynx_quantize_fp8", dev, x, M, K, q.data_ptr(), scale.data_ptr())
    return q, scale


def quantize_fp8_weight(W: torch.Tensor, out: tuple | None = None):
    """The 8-bit operand of a weight (lynx_quantize_fp8_weight).

    Returns (q, scale): q [N, K] float8_e4m3fn and scale [ceil(N/128),
    4 ceil(K/512)] float8_e8m0fnu, the scale of the block of 128 rows x 128
    channels (nb, kb) at scale[nb, kb].  out: the pair of tensors to write.
    """
    N, K, dev, w = _rows(W, torch.bfloat16, "W")
    shape = ((N + 127) // 128, 4 * _scale_words(K))
    if out is None:
        q = torch.empty(N, K, dtype=FP8, device=dev)
        scale = torch.empty(shape, dtype=E8M0, device=dev)
    else:
        q, scale = out
        _expect(q, FP8, (N, K), dev, "q")
        _expect(scale, E8M0, shape, dev, "scale")
    _call("lynx_quantize_fp8_weight", dev, w, N, K, q.data_ptr(), scale.data_ptr())
    return q, scale


def fp8_workspace_bytes(M: int, N: int, K: int) -> int:
    return lib().lynx_fp8_workspace_bytes(M, N, K)


def _fp8_weight(Wq, Ws, K, dev):
    N = Wq.shape[0]
    return (N, _expect(Wq, FP8, (N, K), dev, "Wq"),
            _expect(Ws, E8M0, ((N + 127) // 128, 4 * _scale_words(K)), dev, "Ws"))


def linear_fp8(X, Wq, Ws, Y=None, workspace=None):
    """Y = Q(X) W^T with the weight (Wq, Ws) of quantize_fp8_weight (lynx_linear_fp8)."""
    M, K, dev, x = _rows(X, torch.bfloat16, "X")
    N, wq, ws = _fp8_weight(Wq, Ws, K, dev)
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    else:
        _expect(Y, torch.bfloat16, (M, N), dev, "Y")
    if workspace is None:
        nbytes = fp8_workspace_bytes(M, N, K)
        if nbytes > 0:
            workspace = torch.empty((nbytes,), dtype=torch.uint8, device=dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace: must be a contiguous tensor on {dev}")
    _call("lynx_linear_fp8", dev, x, wq, ws, Y.data_ptr(), M, N, K, _ptr(workspace),
          0 if workspace is None else workspace.numel() * workspace.element_size())
    return Y


def linear_fp8_packed(q, scale, Wq, Ws, Y=None):
    """Y = X W^T of two 8-bit operands, (q, scale) of quantize_fp8 or a block norm
    and (Wq, Ws) of quantize_fp8_weight (lynx_linear_fp8_packed)."""
    M, K, dev, xq = _rows(q, FP8, "q")
    xs = _expect(scale, E8M0, (_scale_words(K), M, 4), dev, "scale")
    N, wq, ws = _fp8_weight(Wq, Ws, K, dev)
    if Y is None:
        Y = torch.empty(M, N, dtype=torch.bfloat16, device=dev)
    else:
        _expect(Y, torch.bfloat16, (M, N), dev, "Y")
    _call("lynx_linear_fp8_packed", dev, xq, xs, wq, ws, Y.data_ptr(), M, N, K)
    return Y


def _sample_rows(t, C, dev, name):
    """(pointer, rows, stride) of per-sample parameters [rows, C] (or [C]); the
    rows may lie apart, as in a slice of a modulation projection's output."""
    shape = t.shape
    if t.dtype is not torch.bfloat16:
        raise TypeError(f"{name}: expected {torch.bfloat16}, got {t.dtype}")
    if not 1 <= len(shape) <= 2 or shape[-1] != C:
        raise ValueError(f"{name}: expected shape (samples, {C}) or ({C},), got {tuple(shape)}")
    if t.device != dev:
        raise ValueError(f"{name}: expected a tensor on {dev}, got one on {t.device}")
    stride = t.stride()
    if stride[-1] != 1:
        raise ValueError(f"{name}: its channels must be contiguous")
    if len(shape) == 1 or shape[0] == 1:
        return t.data_ptr(), 1, 0
    return t.data_ptr(), shape[0], stride[0]


def _block_norm(x, y, gate, post_norm, post_weight, post_bias, post_eps, residual_scale, norm,
                weight, bias, scale, shift, eps, fp8, x_out, out):
    M, C, dev, xp = _rows(x, x.dtype, "x")
    f32 = x.dtype is torch.float32
    if not f32 and x.dtype is not torch.bfloat16:
        raise TypeError(f"x: expected torch.bfloat16 or torch.float32, got {x.dtype}")
    if norm not in NORM_KINDS or post_norm not in NORM_KINDS:
        raise ValueError(f"a norm is one of {list(NORM_KINDS)}")
    rows, bf16 = (M, C), torch.bfloat16
    yp = xo = 0
    if y is not None:
        yp = _expect(y, bf16, rows, dev, "y")
        if x_out is None:
            x_out = torch.empty_like(x)
        xo = _expect(x_out, x.dtype, rows, dev, "x_out")

    def channels(t, name):
        return 0 if t is None else _expect(t, bf16, (C,), dev, name)

    samples = 1
    per_sample = []
    for t, name in ((gate, "gate"), (scale, "scale"), (shift, "shift")):
        if t is None:
            per_sample += 0, 0
            continue
        p, n, stride = _sample_rows(t, C, dev, name)
        if n != 1:
            if samples != 1 and samples != n:
                raise ValueError(f"{name}: {n} samples, and {samples} elsewhere")
            samples = n
        per_sample += p, stride
    gp, gs, sp, ss, hp, hs = per_sample
    h = q = q_scale = 0
    if norm is None:
        if fp8 or out is not None:
            raise ValueError("without a norm there is no second output")
    elif fp8:
        words = _scale_words(C)
        if out is None:
            out = (torch.empty(M, C, dtype=FP8, device=dev),
                   torch.empty(words, M, 4, dtype=E8M0, device=dev))
        else:
            _expect(out[0], FP8, rows, dev, "q")
            _expect(out[1], E8M0, (words, M, 4), dev, "q_scale")
        q, q_scale = out[0].data_ptr(), out[1].data_ptr()
    else:
        if out is None:
            out = torch.empty(M, C, dtype=bf16, device=dev)
        else:
            _expect(out, bf16, rows, dev, "h")
        h = out.data_ptr()
    a = _NORM.pack(xp, yp, gp, channels(post_weight, "post_weight"),
                   channels(post_bias, "post_bias"), channels(weight, "weight"),
                   channels(bias, "bias"), sp, hp, xo, h, q, q_scale, M, C, samples, gs, ss, hs,
                   residual_scale, post_eps, eps, f32, NORM_KINDS[post_norm], NORM_KINDS[norm])
    _call("lynx_block_norm", dev, a)
    return x_out, out


def norm_modulate(x, norm="rms", weight=None, bias=None, scale=None, shift=None, eps=1e-6,
                  fp8=False, out=None):
    """h = norm(x) * (1 + scale[b]) + shift[b], the norm before a block (lynx_block_norm).

    x [M, C] bf16 or fp32; norm "rms" or "layer", with optional weight and bias
    [C]; scale, shift [samples, C] (or [C]), samples of M / samples rows each,
    their rows any multiple of 8 elements apart.  Returns h [M, C] bf16, or with
    fp8=True the 8-bit operand (q, scale) as quantize_fp8 lays it out.
    out: the tensor (or pair) to write.
    """
    if norm is None:
        raise ValueError("norm_modulate needs a norm")
    return _block_norm(x, None, None, None, None, None, 0.0, 1.0, norm, weight, bias, scale, shift,
                       eps, fp8, None, out)[1]


def residual_norm(x, y, gate=None, post_norm=None, post_weight=None, post_bias=None,
                  post_eps=1e-6, residual_scale=1.0, norm=None, weight=None, bias=None, scale=None,
                  shift=None, eps=1e-6, fp8=False, x_out=None, out=None):
    """x' = residual_scale * x + gate[b] * post_norm(y), and the next block's
    h = norm(x') * (1 + scale[b]) + shift[b], in one pass (lynx_block_norm).

    x [M, C] bf16 or fp32 and y [M, C] bf16; the other arguments as in
    norm_modulate, gate [samples, C] (or [C]).  Returns (x', h): x' in x's type
    (x_out may be x), h as norm_modulate returns it, None with norm=None.
    """
    if y is None:
        raise ValueError("residual_norm needs y; use norm_modulate without a branch")
    return _block_norm(x, y, gate, post_norm, post_weight, post_bias, post_eps, residual_scale,
                       norm, weight, bias, scale, shift, eps, fp8, x_out, out)


# dense-equivalent flops of one instruction of each probe kind: smfmac
# 16x16x64, smfmac 32x32x32, mfma 16x16x32, mfma 32x32x16 (bf16)
PROBE_NAMES = ("v_smfmac_f32_16x16x64_bf16", "v_smfmac_f32_32x32x32_bf16",
               "v_mfma_f32_16x16x32_bf16", "v_mfma_f32_32x32x16_bf16")
PROBE_FLOPS = (2 * 16 * 16 * 64, 2 * 32 * 32 * 32, 2 * 16 * 16 * 32, 2 * 32 * 32 * 16)


def probe_mfma_rate(which: int, iters: int, grid: int, device=None) -> dict:
    """Runs lynx_probe_mfma_rate once on torch's current stream and returns the
    event-timed duration with the per-wave stamps (no arithmetic of the layer)."""
    dev = torch.device("cuda") if device is None else device
    sink = torch.empty((grid * 256,), dtype=torch.float32, device=dev)
    stamps = torch.zeros((grid * 4, 2), dtype=torch.int64, device=dev)
    start = torch.cuda.Event(enable_timing=True)
    end = torch.cuda.Event(enable_timing=True)
    start.record()
    _check(lib().lynx_probe_mfma_rate(which, iters, grid, _ptr(sink), _ptr(stamps), _stream(dev)),
           "lynx_probe_mfma_rate")
    end.record()
    torch.cuda.synchronize()
    return {"ms": start.elapsed_time(end), "stamps": stamps.cpu().numpy()}


def probe_mfma(which: int, abid: int, a: torch.Tensor, b: torch.Tensor,
               idx: torch.Tensor | None, d: torch.Tensor) -> torch.Tensor:
    """One matrix instruction per lane on raw register contents (lynx_probe_mfma)."""
    _check(lib().lynx_probe_mfma(which, abid, _ptr(a), _ptr(b), _ptr(idx), _ptr(d),
                                 _stream(a.device)),
           "lynx_probe_mfma")
    return d
