"""GB300 (sm_103a) exact attention: tiled online-softmax prefill, its backward,
paged-KV decode, chunked prefill over the paged cache, rotary positions and
the paged appends that rotate on the way, an 8-bit paged cache with the attention
of single queries, draft tokens and chunks, a 4-bit one with its decode, and the
residual add + RMSNorm and SwiGLU fusions of the same layer.

The compute lives in ``lib/libattn47_sm103.so`` (hand-written CUDA, C-ABI
declared in ``include/attn47.h``); this package is its Python binding.
Importing the package does not load the library; the first call does, and
raises if it is not built.  Build with ``exact_attention_47_gb300.build_lib``.
"""

from ._binding import (  # noqa: F401
    ATTN_DEV_BAD_BLOCK,
    ATTN_DEV_BAD_SEQID,
    ATTN_DEV_BAD_SEQLEN,
    ATTN_DEV_TIMEOUT,
    BLOCK_SIZE,
    AttnError,
    abi_version,
    attn_bwd,
    attn_bwd_workspace_size,
    attn_decode_paged,
    attn_decode_paged_kv4,
    attn_decode_paged_kv4_workspace_size,
    attn_decode_paged_kv8,
    attn_decode_paged_kv8_workspace_size,
    attn_decode_paged_noalloc,
    attn_decode_paged_workspace_size,
    attn_fwd,
    attn_prefill_paged,
    attn_prefill_paged_kv8,
    attn_prefill_paged_kv8_workspace_size,
    device_status,
    fused_add_rmsnorm,
    fused_swiglu,
    kv4_read_paged,
    kv4_record_bytes,
    kv8_append_paged,
    kv8_read_paged,
    kv8_record_bytes,
    library_path,
    load_library,
    rope_append_paged,
    rope_append_paged_kv4,
    rope_bwd,
    rope_fwd,
    selftest_exp2_poly,
    selftest_wait_timeout,
    set_decode_early_plan,
    set_decode_max_ctas,
    set_wait_timeout_ns,
    ssd_chunked_fwd,
    ssd_workspace_size,
    status_string,
    swiglu_projection,
)
