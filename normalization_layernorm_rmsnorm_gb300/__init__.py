"""libnorm for GB300: LayerNorm (rows and channels first), RMSNorm, BatchNorm
(with fused residual and activation), an activation with fused dropout, the
norms and position rotation of attention heads, forward and backward, a
quantised key/value cache with attention over it and eviction from it, and the
norms around a block with its gate and residual scale, as hand-written sm_103a
CUDA kernels behind a C ABI (include/libnorm.h).

This package holds the CUDA sources (``csrc/``), their build (``build.py``),
the ctypes binding of the C ABI (``_binding``, re-exported here under the C
names) and the seeded synthetic input generator (``synth``).
"""
from ._binding import (  # noqa: F401
    ACTS, EXPORTS, KvCache, LIB_PATH, NRM_ACT_ELU, NRM_ACT_GELU, NRM_ACT_LEAKY_RELU, NRM_ACT_MISH,
    NRM_ACT_NONE, NRM_ACT_RELU, NRM_ACT_SILU, NRM_BF16, NRM_CACHE_E4M3, NRM_CACHE_INT4, NRM_CACHE_INT8,
    NRM_ERR_CUDA, NRM_ERR_INVALID_ARG, NRM_ERR_TIMEOUT, NRM_ERR_UNSUPPORTED, NRM_ERR_WORKSPACE, NRM_F16,
    NRM_F32, NRM_OK, NRM_OP_LAYERNORM_BWD, NRM_OP_LAYERNORM_CF_BWD, NRM_OP_QK_NORM_BWD, NRM_OP_RMSNORM_BWD,
    NRM_PAIRS_ADJACENT, NRM_PAIRS_HALF, NrmError, batchnorm_workspace, block_norm_workspace,
    kv_attention_workspace, kv_cache, load, nrm_act_dropout_bwd, nrm_act_dropout_fwd, nrm_act_mask_words,
    nrm_batchnorm_bwd, nrm_batchnorm_fwd,
    nrm_batchnorm_workspace_bytes, nrm_block_norm_bwd, nrm_block_norm_fwd,
    nrm_kv_cache_attention, nrm_kv_cache_evict, nrm_kv_cache_read, nrm_kv_cache_write, nrm_last_error_message,
    nrm_layernorm_bwd, nrm_layernorm_bwd_ex, nrm_layernorm_bwd_noalloc, nrm_layernorm_cf_bwd,
    nrm_layernorm_cf_fwd, nrm_layernorm_fwd, nrm_layernorm_fwd_ex, nrm_qk_norm_rope_bwd,
    nrm_qk_norm_rope_cache, nrm_qk_norm_rope_fwd, nrm_rmsnorm_bwd, nrm_rmsnorm_bwd_ex, nrm_rmsnorm_fwd,
    nrm_rmsnorm_fwd_ex, nrm_rope_bwd, nrm_rope_fwd, nrm_status_str, nrm_sync_status,
    nrm_test_expire_peer_waits, nrm_version, nrm_workspace_bytes, qk_norm_workspace, rope_axis,
)
