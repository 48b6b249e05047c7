"""GB300-native dense fp32 row-major matrix multiplication (SGEMM).

The compute path is the CUDA library ``libsgemm_gb300.so`` built from
``csrc/`` for sm_103a; :mod:`dense_fp32_matrix_major_gb300.sgemm` is its thin
ctypes binding, :mod:`dense_fp32_matrix_major_gb300.experts` the binding of
the mixture-of-experts operators, :mod:`dense_fp32_matrix_major_gb300.fp8` of the
8-bit products and :mod:`dense_fp32_matrix_major_gb300.layer` of the layer for a
few tokens. Importing a binding fails loudly when the library is missing: there is
no CPU fallback.
"""

__all__ = ["experts", "fp8", "layer", "sgemm", "workloads"]
