"""MI355X (gfx950) group-shared fixed fan-in output layer.

The compute lives in libhaste.so (hand-written HIP kernels behind the C ABI
of include/haste.h); ``sparse_output_layer_amd.haste`` is the thin ctypes
binding with the same entry-point names.
"""
from . import haste  # noqa: F401  (fails loudly if libhaste.so is missing)
from .haste import (  # noqa: F401
    Bce, Dropout, HasteError, NormWeights, haste_abi_version, haste_addnorm_bwd,
    haste_addnorm_fwd, haste_dropout_apply, haste_embed_bwd, haste_embed_fwd,
    haste_head_bwd, haste_head_fwd, haste_head_fwd_i8, haste_head_step,
    haste_linear_bwd, haste_linear_fwd, haste_logprob_bwd, haste_logprob_fwd, haste_norm_bwd, haste_norm_fwd,
    haste_quantize_rows, haste_tail_bwd, haste_tail_fwd, haste_tail_group_positives,
    haste_tail_layout, haste_tail_step, haste_tail_validate, haste_topk_merge,
)
