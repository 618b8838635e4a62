"""MI355X (gfx950) GPTQ layer quantizer: Hessian SYRK, damped inverse Cholesky
factor, lazy-block quantize-and-repair, int3/int4 packing, the dequantizing
matrix-vector product over the packed words, the packed product for many tokens
with low-rank adapters beside it and their gradients, the loss over a vocabulary
with its gradients, orthogonalised adapter updates, the Hadamard pre-rotation
and the quantized forward for layer-by-layer calibration, as hand-written HIP
kernels behind the C ABI in include/gptq.h, include/gptq_adapter.h and
include/gptq_train.h."""
from .adapter import adapter_add, adapter_backward, packed_linear, packed_linear_backward
from .gptq import (GPTQError, NotPositiveDefinite, Workspace, dequant_gemv, hadamard_rotate, hessian_accumulate,
                   linear_forward, pack, prepare, prepare_noalloc, quantize_layer, round16)
from .sequential import quantize_mlp_stack
from .train import adapter_orthogonalize, linear_cross_entropy, linear_cross_entropy_backward

__all__ = ["hessian_accumulate", "prepare", "prepare_noalloc", "quantize_layer", "pack", "dequant_gemv", "hadamard_rotate",
           "linear_forward", "round16", "quantize_mlp_stack",
           "packed_linear", "packed_linear_backward", "adapter_add", "adapter_backward",
           "linear_cross_entropy", "linear_cross_entropy_backward", "adapter_orthogonalize", "Workspace",
           "NotPositiveDefinite", "GPTQError"]
