"""GB300 hyper-connection residual read and the verify-window operators beside it: a
C-ABI CUDA library and its Python binding.

``synth`` (seeded inputs) imports without the library. The read itself (``hc_read`` and
friends) and the window operators (``hc_window_plan``, ``hc_kv4_*``,
``hc_token_logprobs``) load ``libhcread.so`` on first use and raise if it is missing:
there is no fallback implementation.
"""
from . import synth  # noqa: F401

_BINDING = ("hc_read_init", "hc_read", "hc_read_path", "hc_read_check", "hc_read_status",
            "hc_read_noalloc", "hc_read_upmix", "hc_read_lo_bf16", "hc_read_y",
            "hc_read_set_wait_limit", "hc_read_bounds_checked",
            "hc_read_shutdown", "hc_read_version", "strerror", "HcReadError", "load",
            "HC_PATH_AUTO", "HC_PATH_DECODE", "HC_PATH_PREFILL", "HC_PATH_PREFILL_UNFUSED",
            "HC_PATH_DECODE_ONE_KERNEL", "HC_PATH_PREFILL_BF16_LO",
            "HC_OK", "HC_ERR_ARG", "HC_ERR_NOT_INIT", "HC_ERR_ARCH", "HC_ERR_CUDA",
            "HC_ERR_TIMEOUT", "HC_ERR_CHECK", "HC_ERR_NOMEM", "HC_ERR_BOUNDS",
            "EXPORTS", "LIB_PATH")

_WINDOW = ("hc_window_plan", "hc_kv4_append", "hc_kv4_load", "hc_kv4_attention",
           "hc_token_logprobs", "hc_kv4_cache", "HC_DTYPE_BF16", "HC_DTYPE_FP16", "HC_DTYPE_FP32",
           "HC_PLAN_MAX_REQUESTS", "HC_KV4_MAX_BLOCK", "HC_KV4_MAX_GROUP", "HC_KV4_MAX_MASKED",
           "HC_LOGPROBS_MAX_TOP", "WINDOW_EXPORTS")


def __getattr__(name):
    if name in _BINDING:
        from . import _lib
        return getattr(_lib, name)
    if name in _WINDOW:
        from . import _window
        return getattr(_window, name)
    raise AttributeError(name)
