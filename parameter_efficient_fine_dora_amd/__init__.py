"""MI355X (gfx950) DoRA hot path: factored row norm, fused compose, backward; and
the operators of a fine-tuning step around it: layer norm, token log
probabilities, AdamW.

The computation lives in libdora.so (HIP kernels behind the C ABI declared in
include/dora.h and include/dora_finetune.h).  ``ops`` is the torch binding with
the same names, ``module`` has the autograd layers and functions, ``optim.AdamW``
the optimizer; they import torch lazily.
"""
from ._lib import LIB_PATH, DoraError, lib  # noqa: F401

__all__ = ["LIB_PATH", "DoraError", "lib"]
