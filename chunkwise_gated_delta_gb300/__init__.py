"""Chunkwise gated delta rule (KDA, GDN, DeltaNet, GLA) on GB300 / sm_103a.

The computation lives in the CUDA library ``_build/libkda.so`` (C ABI in
``include/kda.h``); :mod:`.api` is its Python binding.  The operators around the
mixer (layer norm, short causal convolution, selective scan; ``include/mixer.h``)
are bound by :mod:`.mixer`.  Build the library with
:func:`.build.build`.
"""
from .api import (HostRunner, KdaError, deltanet_fwd, dplr_chunk_bwd, dplr_chunk_fwd, dplr_factor_norms,  # noqa: F401
                  gdn_fwd, gla_fwd, kda_chunk_bwd, kda_chunk_fwd, kda_chunk_fwd_noalloc, status_read)
from .mixer import (layer_norm_bwd, layer_norm_fwd, short_conv_bwd, short_conv_fwd, short_conv_step, ssm_scan_bwd,  # noqa: F401
                    ssm_scan_fwd, ssm_scan_step)
