"""MI355X-native selective scan (Mamba SSM) behind a C-ABI HIP library.

The public entry points mirror the C functions of ``include/ssm_scan.h``:
``ssm_scan_fwd``, ``ssm_scan_fwd_noalloc`` (the same scan without any
allocation), ``ssm_scan_fwd_wavefront`` (the same scan as a chunked
associative scan, for comparison), ``ssm_scan_workspace_size``, ``ssm_scan_aggregate`` (the
affine aggregate of a sequence shard), ``ssm_state_update`` and the backward
pass ``ssm_scan_bwd``; the gated delta rule ``ssm_delta_fwd`` with its decode
window ``ssm_delta_update`` and backward pass ``ssm_delta_bwd``; the head norms with the position rotation,
``ssm_qk_norm_fwd`` and ``ssm_qk_norm_bwd``; the gated linear recurrence ``ssm_glr_fwd`` with
``ssm_glr_update`` and ``ssm_glr_bwd``; and the norms around a block, ``ssm_gated_norm_fwd`` / ``_bwd`` of a
mixer's output with its gate and ``ssm_block_norm_fwd`` / ``_bwd`` between two blocks. They take torch tensors only as carriers of device pointers and the current stream;
every step of the computation runs in the HIP kernels of ``libssmscan.so``.
The library is loaded on first use and a missing build raises at that point.
"""
from .binding import (  # noqa: F401
    SsmError,
    library_path,
    load_library,
    ssm_scan_aggregate,
    ssm_scan_bwd,
    ssm_scan_fwd,
    ssm_scan_fwd_noalloc,
    ssm_scan_fwd_wavefront,
    ssm_scan_workspace_size,
    ssm_state_update,
)
from .binding_delta import (  # noqa: F401
    ssm_delta_bwd,
    ssm_delta_fwd,
    ssm_delta_update,
    ssm_qk_norm_bwd,
    ssm_qk_norm_fwd,
)
from .binding_block import (  # noqa: F401
    ssm_block_norm_bwd,
    ssm_block_norm_fwd,
    ssm_gated_norm_bwd,
    ssm_gated_norm_fwd,
)
from .binding_glr import (  # noqa: F401
    ssm_glr_bwd,
    ssm_glr_fwd,
    ssm_glr_update,
)
