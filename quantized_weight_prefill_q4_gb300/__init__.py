"""GGUF Q4_0 / Q8_0 prefill projections for GB300 (sm_103a).

``Y = X . dequant(W)^T (+ R)``, ``silu(X . Wg^T) * (X . Wu^T)`` and the small-T
GEMV, computed by the hand-written CUDA kernels of ``libapr_qgemm.so``
(C ABI: ``include/apr_qgemm.h``). The names below come from the binding
modules :mod:`quantized_weight_prefill_q4_gb300.capi` and, for the 8-bit KV
cache of the decode steps (``include/apr_kv8.h``),
:mod:`quantized_weight_prefill_q4_gb300.kv8`, loaded on first use so that :mod:`quantized_weight_prefill_q4_gb300.build` can run before the library
exists; using any of them without the built library raises ``ImportError``.
"""


import importlib


def __getattr__(name):
    if name.startswith("__"):
        raise AttributeError(name)
    module = ".kv8" if name.startswith(("apr_kv8_", "Kv8", "KV8_", "APR_T_")) else ".capi"
    try:
        value = getattr(importlib.import_module(__name__ + module), name)
    except AttributeError:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}") from None
    globals()[name] = value  # found at once from now on
    return value
