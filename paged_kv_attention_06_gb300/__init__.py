"""Paged K/V attention for NVIDIA GB300 (sm_103a).

The compute path is the C-ABI library ``_build/libpagedattn.so`` (hand-written
CUDA kernels, declared in ``include/pagedattn.h``); ``binding`` is a thin
ctypes layer with the same entry-point names. Accessing any entry point loads
the library and raises ImportError if it has not been built: there is no CPU
or PyTorch fallback.
"""
_API = ("pa_append_kv", "pa_decode", "pa_prefill", "pa_attention", "pa_attention_route",
        "pa_decode_workspace_bytes", "pa_get_device_error", "status_string", "version",
        "pa_shape", "PagedAttentionError", "decode_workspace", "make_shape",
        "pa_debug_arm_wait_timeout", "pa_debug_prefill_variant", "pa_decode_noalloc",
        "pa_gather_kv", "pa_decode_dense", "KVCache", "KVCacheSnapshot",
        "pa_prefill_split", "pa_prefill_workspace_bytes", "prefill_workspace",
        "pa_append_kv_fp8", "pa_decode_fp8", "pa_prefill_fp8",
        "pa_prefill_fp8_workspace_bytes", "pa_attention_fp8",
        "pa_qk_norm_rope_append", "pa_qk_norm_rope_append_fp8",
        "pa_kv_evict", "pa_kv_evict_fp8", "pa_decode_window", "pa_decode_window_fp8",
        "pa_decode_window_workspace_bytes", "pa_prefill_window", "pa_attention_window", "pa_attention_window_fp8",
        "pa_attention_window_workspace_bytes", "pa_attention_window_fp8_workspace_bytes",
        "pa_decode_weights", "pa_decode_weights_fp8", "pa_decode_weights_workspace_bytes",
        "pa_append_kv_q4", "pa_gather_kv_q4", "pa_decode_q4", "pa_prefill_q4", "pa_attention_q4",
        "pa_decode_q4_workspace_bytes", "pa_prefill_q4_workspace_bytes",
        "pa_attention_q4_workspace_bytes", "pa_decode_prefix", "pa_decode_prefix_fp8",
        "pa_decode_prefix_q4", "pa_decode_prefix_workspace_bytes",
        "pa_decode_prefix_fp8_workspace_bytes", "pa_decode_prefix_q4_workspace_bytes")


def __getattr__(name):
    if name in _API or name.startswith("PA_"):
        from . import binding
        value = getattr(binding, name)
        globals()[name] = value      # found directly from now on
        return value
    raise AttributeError(name)


__all__ = list(_API)
