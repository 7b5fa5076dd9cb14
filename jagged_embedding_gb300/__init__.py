"""GB300-native (sm_103a) jagged index + embedding hot path of FreeScale-style training.

Modules:
  binding   -- ctypes binding of the C ABI (include/fs_jagged.h) over torch tensors
  pipeline  -- one training iteration sequenced over preallocated device buffers
  sequence_block -- the first layer of a sequence model over the gathered rows, with its gradients
  synthetic -- seeded synthetic inputs shaped like the FreeScale workloads
  build     -- in-tree nvcc build of libfsjagged.so
"""
__all__ = ["binding", "pipeline", "sequence_block", "synthetic", "build"]
