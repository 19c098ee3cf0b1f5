"""GB300-native fused flash-attention training op (forward + backward).

The compute path is the C-ABI library libfa_train.so (hand-written sm_103a
CUDA kernels); this package holds its build script, the ctypes binding and
the seeded synthetic workloads used by tests and the benchmark.
"""
from .cache import (cache_evict, cache_read, cache_weights, cache_write, decode, new_cache, prefill)  # noqa: F401
from .fa_train import (FaError, FaParams, bwd, bwd_accum, bwd_accum_rows, bwd_noalloc, bwd_q4, bwd_q8,  # noqa: F401
                       bwd_workspace_size, device_status, fwd, fwd_q4, fwd_q8, fwd_workspace_size, load_library,
                       make_params, set_rows_backward)
from .rope import qk_norm_rope, qk_norm_rope_bwd, rope_inv_freq  # noqa: F401
