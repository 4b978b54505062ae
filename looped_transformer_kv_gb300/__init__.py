"""ResidualQuant decode attention for GB300: librq (C ABI, CUDA sm_103a) + a thin
PyTorch binding.  See include/rq.h for the boundary."""

from .rq import (  # noqa: F401
    PackedCache,
    bf16_decode_attention,
    cache_bytes,
    chunk_attention,
    chunk_workspace_bytes,
    decode_attention,
    decode_workspace_bytes,
    encode_append,
    evict_compact,
    evict_select,
    make_paging,
    make_shape,
    paged_chunk_attention,
    paged_evict_compact,
    res_bits_of,
    synth_params,
    synth_queries,
    synth_states,
)
