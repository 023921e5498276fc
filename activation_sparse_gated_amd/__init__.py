"""Activation-sparse gated FFN for AMD MI355X (gfx950).

The compute path is the HIP library libffn_sparse.so (C ABI in
include/ffn_sparse.h, ffn_gsi.h, ffn_linear.h, ffn_experts.h and ffn_adapter.h); this package only binds
it. Importing works without a GPU; calling an entry point needs the built library and a GPU.
"""
from ._lib import FFNError, load  # noqa: F401
from .adapter import adapter_backward, adapter_forward  # noqa: F401
from .experts import (combine_backward, combine_forward, gather_backward, gather_forward, group_rows,  # noqa: F401
                      route_backward, route_forward)
from .ffn import SparseFFN, TwellPack, moe_forward  # noqa: F401
from .gsi import GsiLinear  # noqa: F401
from .linear import (Fp8Tensor, fp8_linear, fp8_quantize, grouped_backward, grouped_forward,  # noqa: F401
                     rmsnorm_backward, rmsnorm_forward)

__all__ = ["SparseFFN", "TwellPack", "GsiLinear", "moe_forward", "FFNError", "load",
           "Fp8Tensor", "rmsnorm_forward", "rmsnorm_backward", "fp8_quantize", "fp8_linear", "grouped_forward",
           "grouped_backward", "route_forward", "route_backward", "group_rows", "gather_forward", "gather_backward",
           "combine_forward", "combine_backward", "adapter_forward", "adapter_backward"]
