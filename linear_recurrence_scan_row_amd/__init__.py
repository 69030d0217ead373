"""MI355X-native fused affine scans for reinforcement-learning credit assignment.

The seven estimators of the rl-triton summary (GAE, TD(lambda) returns,
discounted returns, V-Trace, Retrace(lambda), eligibility traces, episodic
prefix sums), the generic affine scan over caller-built coefficients, batches
of those calls, and the fused PPO consumers of the advantages (gae_stats,
ppo_clip_loss), each HIP kernel launches behind the C ABI of include/rlca.h.
For policies and models with a recurrent core: the short causal convolution and
the selective state space scan over the same rows, with gradients and
single-step forms, and gradient clipping by the global norm (sequence.py); for a
residual stack of blocks and for generating with it the gated linear recurrence, the
root-mean-square norm with the residual's addition (with gradients, single steps and
an 8-bit output), and a beam search's selection and reordering of states (blocks.py).
recurrent_policy.py trains policies on all of them and plans with one.
Real-valued arrays may be float32, bfloat16 or float16 (fp32 arithmetic).
PyTorch supplies device memory and the stream; the computation is entirely in
librlca.so, which must be built (``python -m linear_recurrence_scan_row_amd.build``).
"""
from .rlca import (  # noqa: F401
    BACKWARD,
    FORWARD,
    Batch,
    RESET_AFTER_DONE,
    RESET_ON_START,
    RlcaError,
    affine_scan,
    discounted_returns,
    eligibility_traces,
    episodic_prefix_sum,
    gae,
    gae_stats,
    gae_stats_noalloc,
    lib,
    ppo_clip_loss,
    retrace,
    td_lambda,
    vtrace,
)
from .sequence import (  # noqa: F401
    ConvGrads,
    ScanGrads,
    causal_conv,
    causal_conv_backward,
    causal_conv_step,
    clip_grad_norm,
    selective_scan,
    selective_scan_backward,
    selective_step,
)
from .blocks import (  # noqa: F401
    BeamChoice,
    GatedGrads,
    NormGrads,
    beam_reorder,
    beam_select,
    gated_recurrence,
    gated_recurrence_backward,
    gated_step,
    rms_norm,
    rms_norm_8bit,
    rms_norm_backward,
)
