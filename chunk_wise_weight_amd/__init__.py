"""MI355X (gfx950) chunk-wise fast-weight update of In-Place Test-Time Training.

The computation lives in libttt.so (hand-written HIP kernels behind a C ABI,
declared in include/ttt.h); this package only binds it. Beside the layer stand
the operators around it: token embedding, the norms between layers with their
gate and residual scales, the plain layers' gated projections and matrix product
with its epilogue, the gradients of all of these, the norm of many gradients
with clipping, and the AdamW step.
"""
from .binding import (  # noqa: F401
    EXPORTS,
    LIB_PATH,
    PHASES,
    GatedGrads,
    Handle,
    LinearGrads,
    NormGrads,
    TTTError,
    lib,
    ttt_adamw,
    ttt_adamw_values,
    ttt_clip_grads,
    ttt_dense_plan,
    ttt_destroy,
    ttt_embed,
    ttt_embed_grad,
    ttt_forward_chunked,
    ttt_forward_chunked_noalloc,
    ttt_forward_docs,
    ttt_gated,
    ttt_gated_grad,
    ttt_init,
    ttt_grad_norm,
    ttt_last_error,
    ttt_linear,
    ttt_linear_grad,
    ttt_phase_times,
    ttt_norm_post,
    ttt_norm_post_grad,
    ttt_norm_pre,
    ttt_norm_pre_grad,
    ttt_plan,
    ttt_reset,
    ttt_set_clip,
    ttt_set_target_conv,
    ttt_set_group_chunks,
    ttt_set_output_f32,
    ttt_set_profiling,
    ttt_state_delta,
    ttt_workspace_bytes,
)
