"""GB300-native DeepSeek-V4 sparse MLA decode attention.

The compute path is the C-ABI library built from ``csrc/`` (CUDA kernels for
sm_103a); ``binding`` marshals torch tensors into that ABI, ``cache`` those
of the paged latent cache.  Importing this package does not load the shared
library; the first call through either does, and raises if it is missing.
"""
__all__ = ["binding", "cache", "workloads"]
