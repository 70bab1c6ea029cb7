"""GB300-native Mamba-2 SSD (state-space duality) chunked selective scan.

The compute lives in ``libssd.so`` (hand-written CUDA for sm_103a behind a
C ABI declared in ``include/ssd.h``); :mod:`state_space_model_mamba_gb300.ssd`
is the thin Python binding that marshals torch tensors into that ABI.
Importing the package loads nothing; the library is opened on first use and
a missing library raises immediately (there is no fallback path).

Beside the scan, with the same conventions: :mod:`mamba3` (``include/mamba3.h``),
:mod:`delta`, the gated delta rule over sequences, its backward and its one-token
step (``include/delta.h``), and :mod:`norm`, the entry norm with the residual's
addition, its e4m3 output and its backward (``include/norm.h``).
"""
__all__ = ["ssd", "mamba3", "delta", "norm", "inputs"]
