"""fine_grained_fp8_persistent_gb300 -- fine-grained FP8 NT GEMM engine for GB300.

The compute lives in libfgf8.so (hand-written sm_103a CUDA kernels behind the C
ABI in include/fgf8.h).  The names below come from ``binding`` and are loaded on
first use, so ``fine_grained_fp8_persistent_gb300.inputs`` (seeded synthetic
inputs) can be imported on machines where the library is not built.
"""
from __future__ import annotations

_EXPORTS = (
    "quantize_1x128", "quantize_128x128", "gemm_f16", "gemm_fp8_blockscaled", "gemm_fp8_blockscaled_quant",
    "grouped_fp8_contiguous", "grouped_fp8_masked", "check_status",
    "mk_alignment_for_contiguous", "sfa_bytes", "sfb_bytes", "sfa_shape", "sfb_shape",
    "set_wait_timeout_ms", "set_pdl", "selftest_wait_timeout", "last_error", "last_tile", "version", "FGF8Error", "SCALE_F32", "SCALE_UE8M0",
    "quantize_fp4", "gemm_fp4_blockscaled", "fp4_sf_shape", "FP4_MX", "FP4_NV",
    "gated_f16", "gated_f16_backward", "gated_backward_ws_bytes", "gemv_fp4", "gated_gemv_fp4", "GEMV_MAX_ROWS",
    "ACT_SILU", "ACT_GELU_TANH",
    "Route", "route_contiguous", "route_masked", "route_rows", "dispatch_f16", "dispatch_fp8", "dispatch_f16_backward",
    "combine_f16", "combine_f16_backward", "lora_f16",
)


_NAMES = frozenset(_EXPORTS)
_binding = None


def __getattr__(name):
    # looked up in binding at every use, so that what is replaced there is replaced here
    # (0.4 us; an import statement each time makes it 1 us)
    global _binding
    if name in _NAMES:
        if _binding is None:
            from . import binding as _binding
        return getattr(_binding, name)
    raise AttributeError(name)


__all__ = list(_EXPORTS)
