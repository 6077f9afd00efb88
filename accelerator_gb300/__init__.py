"""accelerator_gb300 -- libgemm, dense C = A*B on one GB300 (sm_103a).

The compute lives in the CUDA library built from ``csrc/`` (see ``build.py``);
``binding.py`` is the thin ctypes layer over its C ABI, ``lowbit.py`` the one
over its operators on operands held in 4 or 8 bits.  Importing the package
loads nothing: the library is opened at the first call, and a missing library
is an error, never a fallback.
"""

FP32, TF32, BF16, FP16, FP32_VIA_BF16 = 0, 1, 2, 3, 4

__all__ = ["gemm", "gemm_ex", "GemmError", "FP32", "TF32", "BF16", "FP16", "FP32_VIA_BF16",
           "W4Matrix", "w4_quantize", "w4_dequantize", "gemm_w4", "KvCache", "kv_append", "kv_read",
           "kv_attention"]

_LOWBIT = __all__[8:]


def __getattr__(name):
    if name in ("gemm", "gemm_ex", "GemmError"):
        from . import binding
        return getattr(binding, name)
    if name in _LOWBIT:
        from . import lowbit
        return getattr(lowbit, name)
    raise AttributeError(name)
