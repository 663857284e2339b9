"""GB300-native deterministic sparse top-k and sparse MLA attention.

The compute lives in hand-written sm_103a CUDA kernels behind the C ABI of
``include/ds_sparse_mla.h`` (``libds_sparse_mla.so``, built in-tree by
``invariant_sparse_mla_gb300.build``). This package only marshals torch
tensors and the current stream into those calls.
"""

from ._native import (  # noqa: F401
    DSError,
    DEVERR_IDX,
    DEVERR_LEN,
    DEVERR_NOPAGE,
    DEVERR_PAGE,
    DEVERR_ROWREQ,
    DEVERR_SHARED,
    DEVERR_TIMEOUT,
    EXPORTED,
    attention_workspace_size,
    indexer_logits,
    kv_cache_write,
    last_error,
    lib,
    sparse_mla_decode,
    sparse_mla_decode_swa,
    sparse_mla_prefill,
    supported_config,
    swa_workspace_size,
    topk_per_row,
    topk_workspace_size,
)
from .kv8 import (  # noqa: F401
    kv8_accept,
    kv8_append,
    kv8_decode,
    kv8_decode_workspace_size,
    kv8_evict,
    kv8_evict_workspace_size,
    kv8_mass,
    kv8_prefill,
    kv8_prefill_workspace_size,
    kv8_tree_decode,
    kv8_tree_decode_workspace_size,
)
from .norm_rope import qk_norm_rope  # noqa: F401
from .pages import (  # noqa: F401
    pages_compact,
    pages_copy,
    pages_extend,
    pages_fork,
    pages_free,
    pages_shrink,
    pages_workspace_size,
)
