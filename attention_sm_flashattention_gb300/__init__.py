"""GB300 FlashAttention: exact tiled attention forward and backward for sm_103a.

``fwd``/``bwd`` call the C ABI of ``libfa.so`` (built in-tree by
``attention_sm_flashattention_gb300.build``).  The library is loaded on the
first call; if it is missing the call raises -- there is no other path.
"""

from .api import bwd, bwd_flops, bwd_workspace_size, device_status, fwd, fwd_flops, fwd_paged, fwd_sparse, paged_split_count, reshape_and_cache  # noqa: F401
from .scored import KeyRanges, bwd_scored, fwd_paged_scored, fwd_scored, key_ranges, rotary, rotary_and_cache, rotary_axes, rotary_bwd, rotary_freqs  # noqa: F401
from .paging import cache_release, cache_step, page_pool  # noqa: F401
