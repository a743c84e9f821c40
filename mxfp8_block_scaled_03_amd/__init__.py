"""MI355X (gfx950) MXFP8 and MXFP4 library: OCP-MX block-scaled quantize, dequantize and GEMM,
and a mixture-of-experts layer with MXFP4 weights.

The compute path is the HIP library ``libmxq.so`` built from ``csrc/`` (C ABI in
``include/mxq.h``).  This package only marshals arguments: the ``mxq_*`` functions
mirror the C entry points one to one (plain integers and device pointers), and
``quantize`` / ``dequantize`` / ``gemm`` are torch-tensor conveniences that allocate
outputs with torch and call them on torch's current stream; the ``*_fp4`` functions
(``_fp4.py``, loaded on first use) are theirs for MXFP4.  There is no fallback:
if the library is missing, every call raises.

Sources: "Low-Precision GPU Programming" -- "Scale ownership and the GEMM dataflow"
(Y = XW, block scales inside the K sum), "Microscaling: the two-row experiment" (32-element
blocks, E8M0 scales, conservative power-of-two scale rule), "Hardware support and kernel
ABI contracts" (dtype tags, scales, orientation and padding travel together).
"""
from ._binding import (  # noqa: F401
    MXQ_ACC_FP32, MXQ_ACC_FP8_MFMA, MXQ_ACT_NONE, MXQ_ACT_SILU, MXQ_BF16, MXQ_COLWISE, MXQ_E2M1, MXQ_E4M3, MXQ_E5M2,
    MXQ_F32, MXQ_ROWWISE, MXQ_SCALE_CEIL, MXQ_SCALE_OCP, MxqError, dequantize, gemm, lib, library_path,
    mxq_dequantize, mxq_gemm, mxq_gemm_ex, mxq_gemm_ex_noalloc, mxq_quantize, mxq_quantize_dual, mxq_quantize_rule, mxq_quantize_scaled,
    mxq_dequantize_fp4, mxq_gemm_exact_plan, mxq_gemm_fp4, mxq_gemm_fp4_plan, mxq_moe_fp4, mxq_moe_fp4_plan,
    mxq_moe_fp4_workspace, mxq_quantize_fp4, mxq_quantize_fp4_dual, mxq_quantize_fp4_sr, mxq_quantize_sr, mxq_status_string, mxq_version,
    quantize, quantize_dual, quantize_scaled, quantize_sr,
)

_FP4 = ("dequantize_fp4", "gemm_fp4", "moe_fp4", "quantize_fp4", "quantize_fp4_dual", "quantize_fp4_sr")


def __getattr__(name):
    # the torch conveniences import torch with their module, which the raw entry points do not need
    if name in _FP4:
        from . import _fp4
        value = globals()[name] = getattr(_fp4, name)
        return value
    raise AttributeError("module %r has no attribute %r" % (__name__, name))
