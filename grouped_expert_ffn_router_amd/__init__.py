"""MI355X-native fixed-pool, three-wave MoE expert layer (one EP rank).

The layer runs in libmoe.so (hand-written HIP kernels for gfx950 behind the C
ABI of include/moe.h).  ``binding`` marshals arguments into that ABI and
``runner`` lays out device buffers with torch; neither computes any part of
the layer.  ``block`` has the operators around the experts' products (norm,
choice of experts, SwiGLU with an 8-bit checkpoint, MX-FP8 rows) on torch
tensors, ``training`` the same under torch's autograd.
"""

from . import binding  # noqa: F401

__all__ = ["binding"]
