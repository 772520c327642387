"""MI355X-native GGUF Q4_0 weight-only linear layer, and the decoder operators
between the linears.

The computation lives in libq4amd.so (HIP kernels for gfx950 behind the C ABI
of include/q4_0.h, include/q4_decoder.h and include/q4_search.h); this package is its thin Python binding.
The library is loaded on first use and a missing build raises instead of falling back.
"""

from ._binding import (  # noqa: F401
    EXPORTS,
    PackedWeight,
    Q4Error,
    dequant,
    embed,
    embed_gguf,
    gguf_bytes,
    lib,
    library_path,
    linear,
    linear_kernel,
    linear_multi,
    linear_swiglu,
    linear_swiglu_kernel,
    pack,
    packed_bytes,
    quantize,
    PackedWeightQ41,
    q41_dequant,
    q41_linear,
    q41_linear_kernel,
    q41_pack,
    q41_packed_bytes,
    q41_quantize,
    reference_mfma,
    reference_read,
    status_str,
    time_next_launch,
    unpack,
)
from ._decoder import (  # noqa: F401
    DECODER_EXPORTS,
    KV_BLOCK,
    KVCache,
    add_rmsnorm,
    kv_append,
    kv_attention,
    kv_attention_plan,
    kv_attention_workspace,
    kv_cache_bytes,
    logits_adjust,
    rope_table,
)
from ._search import (  # noqa: F401
    SEARCH_EXPORTS,
    KVCompact,
    KVFork,
    KVStack,
    beam_advance,
    beam_select,
    beam_select_workspace,
    kv_attention_blocks,
    kv_attention_blocks_workspace,
    kv_compact,
    kv_compact_workspace,
    kv_copy_blocks,
    kv_fork,
    kv_fork_workspace,
    kv_select,
    kv_select_workspace,
    kv_summarize,
    kv_summary,
)
