"""GB300 (sm_103a) passes of chunkwise gated linear attention, of the gated delta rule and of the selective scan, and of
what stands around them in a layer: the short causal convolution, the norms and rotation of the queries and
keys, the heads' norm with its gate, the residual with its norm.

The compute lives in libgla.so (C ABI, include/gla.h); ``binding`` is the
ctypes layer over it with the same names. Importing this package does not
load the library; the first call does, and raises if it is not built.
"""
from .binding import (  # noqa: F401
    GLA_BF16, GLA_FP32, GLA_GATE_BILINEAR, GLA_GATE_HEAD_SCALAR, GLA_GATE_NONE, GLA_GATE_PER_KEY,
    GLA_GATE_TOKEN_SCALAR,
    GLA_PATH_AUTO, GLA_PATH_FUSED, GLA_PATH_SIMT, GLA_PATH_SPLIT, GLA_PATH_STAGED, GLA_PATH_TENSOR, GlaError,
    backward, forward, gla_bwd,
    gla_bwd_num_stages, gla_bwd_stage, gla_bwd_stage_name, gla_bwd_workspace_size, gla_device_status,
    gla_fwd, gla_fwd_ex, gla_fwd_host, gla_fwd_num_stages, gla_fwd_stage, gla_fwd_stage_name,
    gla_fwd_workspace_size, gla_host_release, gla_pair_combine, gla_pair_scan, gla_segment_pair,
    gla_segment_pair_workspace_size, gla_status_string, gla_version, make_params, pair_combine, pair_scan,
    segment_pair,
    GLA_NORM_L2, GLA_NORM_NONE, GLA_NORM_RMS, delta_backward, delta_forward, gla_delta_bwd,
    gla_delta_bwd_workspace_size, gla_delta_fwd, gla_delta_fwd_workspace_size, gla_qk_norm_rope,
    gla_qk_norm_rope_bwd, gla_qk_norm_rope_bwd_workspace_size, qk_norm_rope_backward, qk_norm_rope_forward,
    GLA_ACT_NONE, GLA_ACT_SIGMOID, GLA_ACT_SILU, causal_conv_backward, causal_conv_forward, gla_conv_bwd,
    gla_conv_bwd_workspace_size, gla_conv_fwd, gla_norm_gate, gla_norm_gate_bwd, gla_norm_gate_bwd_workspace_size,
    gla_residual_norm, gla_residual_norm_bwd, gla_residual_norm_bwd_workspace_size, gla_ssm_bwd,
    gla_ssm_bwd_workspace_size, gla_ssm_fwd, gla_ssm_fwd_workspace_size, norm_gate_backward, norm_gate_forward,
    residual_norm_backward, residual_norm_forward, selective_scan_backward, selective_scan_forward,
)
from .autograd import (  # noqa: F401,E402
    causal_conv, delta_attention, gla_attention, norm_gate, qk_norm_rope, residual_norm, selective_scan,
)
