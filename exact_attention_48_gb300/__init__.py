"""GB300-native exact attention: fa_fwd / fa_bwd over a C-ABI CUDA library.

Importing the package is cheap; the shared library (``libfa.so``) is loaded
on first use and the import fails loudly when it is missing.  There is no
CPU fallback.
"""
from .binding import (  # noqa: F401
    FaError,
    fa_bwd,
    fa_bwd_strided,
    fa_bwd_varlen,
    fa_bwd_workspace_bytes,
    fa_decode_workspace_bytes,
    fa_device_status,
    fa_fwd,
    fa_fwd_decode,
    fa_fwd_fp8,
    fa_fwd_strided,
    fa_fwd_varlen,
    library,
    status_string,
)
from .cache_ops import (  # noqa: F401
    fa_cache_compact,
    fa_cache_select,
    fa_fwd_tree,
    fa_key_weights,
    fa_key_weights_workspace_bytes,
    fa_rope,
    fa_rope_append,
    fa_rope_bwd,
    fa_rope_frequencies,
    fa_tree_workspace_bytes,
)
from .cache8_ops import (  # noqa: F401
    fa_cache_compact_fp8,
    fa_fwd_tree_fp8,
    fa_rope_append_fp8,
    fa_tree_fp8_workspace_bytes,
    fa_tree_verify,
)
