"""MI355X (gfx950) selective state-space scan (S6): fused scan forward, its
backward (gradients by state recomputation) and one-token decode, and the causal convolution + SiLU front-end of the SSM
branch, as hand-written HIP kernels behind a C ABI (``include/mamba_scan.h``,
``include/mamba_scan_bwd.h``, ``include/mamba_conv.h``), with a thin ctypes binding;
and the Mamba-2 SSD layer by the chunked algorithm on the matrix cores
(``include/mamba_ssd.h``). Around them, the operators of a recurrent block
(``include/block/``): the gated linear recurrence (sequences, backward, decode
token), the RMS norm with the residual's addition (io or 8-bit output,
backward) and the convolution's backward; and those of a matrix-state mixer
(``include/mixer/``): linear attention with a decay for each head (sequences,
backward, decode token) and the norm and position rotation of its queries and
keys.

``scan_fwd`` and ``state_update`` call the native library; importing this
package does not load it, but the first call does, and raises if the library
has not been built (there is no fallback path).
"""
from .block import (conv1d_bwd, gated_scan_bwd, gated_scan_fwd, gated_update,  # noqa: F401
                    rmsnorm_bwd, rmsnorm_fwd, rmsnorm_quant_fwd)
from .binding import (bwd_workspace_size, conv1d_fwd, conv1d_update, library_path,  # noqa: F401
                      load_library, scan_bwd, scan_fwd, ssd_fwd, state_update, workspace_size)
from .mixer import (linear_attn_bwd, linear_attn_fwd, linear_attn_update, qk_norm_rope_bwd,  # noqa: F401
                    qk_norm_rope_fwd)
