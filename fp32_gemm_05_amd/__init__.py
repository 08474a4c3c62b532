"""libsgemm: single-precision GEMM (C = alpha*op(A)*op(B) + beta*C, row-major fp32) for MI355X.

The compute path is hand-written HIP for gfx950 behind a C ABI
(``include/sgemm.h``, ``libsgemm.so``); this package is the thin ctypes binding
over it.  Importing the package loads nothing: the shared library is opened on
the first call, and a missing library raises instead of falling back to any
other implementation.

``vocab_*`` are the vocabulary-head operators (``include/vocab.h``; cross entropy and distillation
over X @ W.T without keeping the logits), in ``vocab.py``, which is imported at their first use.
"""
from ._binding import (  # noqa: F401
    SgemmArgumentError,
    SgemmError,
    SgemmLaunchError,
    gemm,
    library_path,
    load_library,
    sgemm,
    sgemm_ex,
    sgemm_last_variant,
    sgemm_num_variants,
    sgemm_op,
    sgemm_op_ex,
    sgemm_op_select_variant,
    sgemm_select_variant,
    sgemm_variant_info,
    sgemm_variant_name,
    sgemm_version,
    tile_order,
)

_VOCAB = ("vocab_ce", "vocab_ce_grad", "vocab_distill", "vocab_distill_grad", "vocab_workspace",
          "vocab_cross_entropy", "vocab_distillation")


def __getattr__(name):
    if name not in _VOCAB:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    from . import vocab
    globals().update({n: getattr(vocab, n) for n in _VOCAB})
    return globals()[name]
