"""GB300 (sm_103a) mixture-of-experts layer: routing, int4 grouped expert GEMMs and
decode; grouped-query decode attention over a fixed-block KV cache; a KV cache
in 4- or 8-bit codes (append, read back, decode and prefill attention); the
Gated DeltaNet scan; and what lies between them in a serving step: norms, 4-bit
matrix-vector products, rotary positions and the verification of drafted tokens.

The compute lives in liblily_moe.so (CUDA kernels behind a C ABI, see
include/lily_moe.h); ``_abi`` is its ctypes binding.  Importing this package
loads nothing; the library is built / loaded on first use.
"""
from ._abi import (alloc_draft_workspace, lily_draft_verify, lily_q4_matvec, lily_rms_norm, lily_rope, make_q4,  # noqa: F401
                   make_rope_table, rope_frequencies)
from ._abi import (LilyError, alloc_attn_workspace, alloc_kvq_cache, alloc_kvq_workspace, lily_kvq_append,  # noqa: F401
                   lily_kvq_attn_decode, lily_kvq_attn_prefill, lily_kvq_read, lily_kvq_workspace_bytes,
                   make_kvq_cache, make_kvq_shape, alloc_routing, lily_attn_decode, lily_attn_workspace_bytes,  # noqa: F401
                   make_attn_shape, lily_gdn_scan, alloc_workspace, lily_moe_block_capacity, lily_moe_check_shape,  # noqa: F401
                   lily_moe_clear_status, lily_moe_decode, lily_moe_device_status, lily_moe_forward,
                   lily_moe_forward_timed, lily_moe_grouped_gemm, lily_moe_last_error_detail, lily_moe_route, lily_moe_route_noalloc, lily_moe_status_string,
                   lily_moe_version, lily_moe_workspace_bytes, load, make_routing, make_shape, make_weights)
