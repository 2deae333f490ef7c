"""B200-native (sm_100a) fused per-token normalisation cores of the Muse Spark
Open decoder layer, behind the C ABI declared in include/muse_cores.h.

    from gate_cores_b200 import rms_norm, input_scale_norm, qk_norm_rope, \\
        output_norm_gate, norm_residual

and, beside them, the other per-token steps of a layer: layer norm, rotary positions, and the rows of tokens to their
experts and back.

Every call runs in libmuse_cores.so (built by ``python -m gate_cores_b200.build``);
without the library the first call raises - there is no CPU fallback.
"""
from ._lib import MuseError, load as load_library  # noqa: F401
from .cores import (  # noqa: F401
    expert_combine,
    expert_combine_backward,
    expert_dispatch,
    expert_dispatch_backward,
    expert_sort,
    input_scale_norm,
    layer_norm,
    layer_norm_backward,
    norm_residual,
    output_norm_gate,
    qk_norm_rope,
    residual,
    residual_blend,
    residual_gate_angles,
    rms_norm,
    rope,
    rope_backward,
    rope_frequencies,
    stream_copy,
)

__all__ = ["rms_norm", "input_scale_norm", "qk_norm_rope", "output_norm_gate", "norm_residual",
           "residual_blend", "residual", "residual_gate_angles", "layer_norm", "layer_norm_backward", "rope",
           "rope_backward", "rope_frequencies", "expert_sort", "expert_dispatch", "expert_dispatch_backward",
           "expert_combine", "expert_combine_backward", "stream_copy", "MuseError", "load_library"]
