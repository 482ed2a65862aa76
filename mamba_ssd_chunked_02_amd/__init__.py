"""MI355X-native Mamba-2 SSD chunked scan (forward and backward).

The compute runs in ``libssd.so`` (HIP kernels for gfx950 behind the C ABI
of ``include/ssd.h``); this package is its Python binding.  Functions carry
the C names: ``ssd_fwd``, ``ssd_fwd_workspace_bytes``, ``ssd_status_string``,
``ssd_abi_version``, ``ssd_fwd_plan``, ``ssd_fwd_ex`` (as
``prepare(..., tuning=...).run(stages)``), ``ssd_bwd``, ``ssd_bwd_ex``,
``ssd_bwd_workspace_bytes`` (``prepare_bwd(...).run()`` re-launches);
``ssd_fwd_bidir`` (``prepare_bidir(...).run()`` re-launches) runs both
directions of the bidirectional mode.

The operators around the scan: ``ssd_norm_fwd`` / ``ssd_norm_bwd`` (layer
norm), ``ssd_conv_fwd`` / ``ssd_conv_bwd`` (short causal convolution with
SiLU), ``ssd_selscan_fwd`` / ``ssd_selscan_bwd`` (selective scan with a decay
per channel and state entry), and for serving one token at a time
``ssd_step``, ``ssd_conv_step`` and ``ssd_selscan_step``.  Linear attention with
a constant decay per head: ``ssd_linattn_fwd`` / ``ssd_linattn_bwd`` and
``ssd_linattn_step`` for single tokens.  ``ssd_groupnorm_fwd`` /
``ssd_groupnorm_bwd``: group norm, channels last, with SiLU or a gate.
"""
from ._binding import (  # noqa: F401
    CHUNK, SSD_BF16, SSD_F32, STAGE_ALL, STAGE_PASS, STAGE_SCAN, STAGE_STATE, STAGE_TABLE,
    TUNING_FIELDS, PreparedBidir, PreparedBwd, PreparedCall, SsdDims, SsdError, SsdLayout, SsdPlanInfo,
    SsdTuning, dims_for, layout_of, library, make_dims, make_tuning, prepare, prepare_bidir, prepare_bwd,
    ssd_abi_version, ssd_bwd, ssd_bwd_workspace_bytes, ssd_fwd, ssd_fwd_bidir, ssd_fwd_noalloc,
    ssd_fwd_noalloc_max_bytes, ssd_fwd_plan,
    ssd_fwd_workspace_bytes, ssd_status_string,
)
from ._layer import (  # noqa: F401
    SsdConvDims, SsdConvLayout, SsdGroupnormDims, SsdLinattnDims, SsdLinattnLayout, SsdNormDims, SsdSelscanDims,
    SsdSelscanLayout, ssd_conv_bwd, ssd_conv_fwd, ssd_conv_step, ssd_groupnorm_bwd,
    ssd_groupnorm_fwd, ssd_linattn_bwd, ssd_linattn_fwd,
    ssd_linattn_step, ssd_norm_bwd, ssd_norm_fwd, ssd_selscan_bwd, ssd_selscan_fwd,
    ssd_selscan_step, ssd_step,
)
