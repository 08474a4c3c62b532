"""libsgemm: single-precision GEMM (C = alpha*op(A)*op(B) + beta*C, row-major fp32) for MI355X.

The compute path is hand-written HIP for gfx950 behind a C ABI
(``include/sgemm.h``, ``libsgemm.so``); this package is the thin ctypes binding
over it.  Importing the package loads nothing: the shared library is opened on
the first call, and a missing library raises instead of falling back to any
other implementation.

``vocab_*`` are the vocabulary-head operators (``include/vocab.h``; cross entropy and distillation
over X @ W.T without keeping the logits), in ``vocab.py``, which is imported at their first use.  So are
``linear_*`` (a linear layer with bias, activation and residual; ``include/linear.h``), ``vocab_sample`` (drawing
tokens from logits; ``include/sample.h``), ``grad_norm`` and ``clip_grad_norm`` (``include/grads.h``).
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

# the operators' modules, imported at the first use of one of their names
_OPERATORS = {
    "vocab": ("vocab_ce", "vocab_ce_grad", "vocab_distill", "vocab_distill_grad", "vocab_workspace",
              "vocab_cross_entropy", "vocab_distillation"),
    "linear": ("linear_act", "linear_act_grad", "linear_workspace", "linear_layer"),
    "sample": ("vocab_sample", "vocab_sample_workspace"),
    "grads": ("grad_norm", "clip_grad_norm", "grad_workspace"),
}
_MODULE_OF = {name: module for module, names in _OPERATORS.items() for name in names}


def __getattr__(name):
    if name not in _MODULE_OF:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    import importlib
    module = importlib.import_module("." + _MODULE_OF[name], __name__)
    globals().update({n: getattr(module, n) for n in _OPERATORS[_MODULE_OF[name]]})
    return globals()[name]
