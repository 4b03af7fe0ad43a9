"""EXL3 trellis-quantized linear layer for GB300 (sm_103a).

The compute lives in ``libexl3.so`` (hand-written CUDA behind a C ABI, see
``include/exl3.h``).  This package is a thin binding: it marshals torch
tensors into pointers and sizes and calls the library.  There is no CPU or
PyTorch fallback; if the library is missing every call raises.

Beside the layer: rotary positions (``rope``), a paged cache of 16, 8 or 4 bits
(``KVCache``, ``kv_write``, ``kv_read``) and attention over prompts
(``attention_prompt``) and over the cache (``attention_paged``).
"""
from .binding import (  # noqa: F401
    CODEBOOKS,
    KV_FORMATS,
    Exl3Error,
    KVCache,
    attention_paged,
    attention_paged_workspace_bytes,
    attention_prompt,
    autotune_entries,
    clear_autotune,
    device_status,
    gemm,
    gemm_splitk,
    input_transform,
    input_transform_swiglu,
    kv_read,
    kv_write,
    lib,
    linear,
    set_autotune,
    moe_combine,
    moe_gemm,
    moe_input_transform,
    rope,
    rope_phases,
    splitk_parts,
    splitk_workspace_bytes,
    status_string,
    test_codebook,
    test_unpack,
)
