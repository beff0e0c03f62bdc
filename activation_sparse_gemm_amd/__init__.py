"""RT-Lynx sparse + LoRA linear layer on AMD MI355X (gfx950).

Python face of liblynx.so: `sparsify`, `linear_sparse_lora`,
`linear_sparse_lora_packed`, `linear_sparse_lora_noalloc`, `linear_dense`, the
8-bit layer (`quantize_fp8`, `quantize_fp8_weight`, `linear_fp8`,
`linear_fp8_packed`), the block norms (`norm_modulate`, `residual_norm`), rotary
positions (`qk_rotary`) and `attention` take torch device tensors and call the
library's HIP kernels on torch's current stream.
"""
from ._abi import (  # noqa: F401
    LIB_PATH,
    SCRATCH_BYTES,
    LynxError,
    attention,
    attention_workspace_bytes,
    fp8_workspace_bytes,
    lib,
    linear_dense,
    linear_fp8,
    linear_fp8_packed,
    linear_sequence,
    sequence_workspace_bytes,
    linear_sparse_lora,
    linear_sparse_lora_noalloc,
    linear_sparse_lora_packed,
    norm_modulate,
    qk_rotary,
    quantize_fp8,
    quantize_fp8_weight,
    residual_norm,
    sparsify,
    status_string,
    version,
    workspace_bytes,
)
