"""GB300-native exact attention forward (sm_103a).

The compute lives in a C-ABI CUDA library (``libattn_sm103.so``, declared in
``include/attn.h``); ``_native`` only marshals arguments to it.
"""
from ._native import (  # noqa: F401
    ATTN_OK,
    AttnError,
    attn_fwd,
    attn_fwd_splitkv,
    attn_get_device_status,
    attn_splitkv_workspace_size,
    attend_blocks_paged,
    decode,
    decode_paged_fp8,
    decode_paged_shared,
    forward,
    kvcache_append_paged,
    kvcache_append_paged_fp8,
    kvcache_bounds_paged,
    kvcache_release_paged,
    kvcache_reserve_paged,
    qk_norm_rope,
    qk_norm_rope_bwd,
    rope_table,
    select_blocks_paged,
    status_string,
)
