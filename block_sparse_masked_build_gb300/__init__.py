"""GB300-native block-sparse masked attention (Splash-style): forward and
backward, with a tanh cap and a distance bias of the scores where wanted, and
a paged 8-bit key/value cache with the attention that reads it.

The compute runs in libbsm.so (hand-written CUDA for sm_103a) behind the C
ABI of ``include/bsm.h``; this package is its Python binding.
"""

from .api import (  # noqa: F401
    MASK_BAND,
    MASK_CAUSAL,
    MASK_DENSE,
    MASK_LOCAL,
    MASK_SEGMENT,
    SCORE_POINTWISE,
    SCORE_SOFTMAX,
    BsmError,
    KVCache,
    MaskInfo,
    bsm_build_mask_info,
    bsm_device_status,
    bsm_kv_append,
    bsm_last_error,
    bsm_mask_info_bytes,
    bsm_pack_dense_mask,
    bsm_paged_attention,
    bsm_paged_attention_workspace_bytes,
    bsm_selftest_wait_timeout,
    bsm_splash_bwd,
    bsm_splash_bwd_mod_workspace_bytes,
    bsm_splash_bwd_workspace_bytes,
    bsm_splash_fwd,
    bsm_splash_fwd_host,
    bsm_splash_fwd_host_bytes,
    bsm_splash_fwd_workspace_bytes,
    bsm_version,
    build_mask_info,
    kv_append,
    pack_dense_mask,
    paged_attention,
    splash_attention,
    splash_attention_bwd,
)
