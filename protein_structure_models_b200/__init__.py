"""Fused Invariant Point Attention forward for B200 (sm_100a).

The compute lives in libfipa.so (C ABI in include/fipa.h); this package is
its thin Python binding and build step."""
from .fipa import (Fipa, FipaError, FipaDims, embedding, embedding_backward,  # noqa: F401
                   embedding_backward_workspace_size, invariant_point_attention, load_library,
                   library_path, make_dims, norm_residual, norm_residual_backward)
