"""B200 (sm_100a) WAITS prefill KV-eviction path: score -> select -> compact.

The work runs in ``libwaits.so`` (hand-written CUDA kernels behind a C ABI,
``include/waits.h``); :mod:`.api` marshals torch tensors into it.  Importing
this package does not load the library; the first call does, and raises if
it is missing (there is no fallback).
"""

from .api import (  # noqa: F401
    Compressor, HostCompressor, compact, compress, score, score_static, select,
    select_compact,
    workspace_bytes, make_shape)
from .cache import (  # noqa: F401
    Q4Cache, cache_release, cache_reserve, q4_append, q4_compact, q4_decode_attention,
    q4_decode_workspace_bytes, q4_page_bytes, q4_read, qk_norm_rope, rotary_inv_freq)
from ._lib import WaitsError, WaitsLibraryError  # noqa: F401
