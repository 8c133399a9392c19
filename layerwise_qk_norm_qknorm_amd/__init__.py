"""Layerwise QK-Norm for MI355X (gfx950): HIP kernels behind a small C ABI.

The compute lives in ``libqknorm.so`` (built from ``csrc/``); this package is
argument marshalling only. Importing it does not load the library; the first
call does, and raises if the library has not been built.
"""

from .binding import (  # noqa: F401
    PreparedCall,
    QKNormError,
    abi_version,
    describe_headwise_plan,
    describe_plan,
    library_path,
    load_library,
    qknorm_apply_with_stats,
    qknorm_fused,
    qknorm_headwise,
    qknorm_partial_stats,
    prepare_apply_with_stats,
    prepare_fused,
    prepare_headwise,
    prepare_partial_stats,
)

_OPERATORS = ("prepare_headwise_rope", "prepare_headwise_rope_axes", "prepare_headwise_rope_axes_backward",
              "prepare_headwise_rope_backward", "prepare_paged_append", "prepare_paged_append_axes",
              "prepare_paged_attend", "prepare_paged_attend_wide", "prepare_paged_gather", "qknorm_headwise_rope",
              "qknorm_headwise_rope_axes", "qknorm_headwise_rope_axes_backward", "qknorm_headwise_rope_backward",
              "qknorm_paged_append", "qknorm_paged_append_axes", "qknorm_paged_attend", "qknorm_paged_attend_wide",
              "qknorm_paged_gather", "rope_axes", "rope_table")


def __getattr__(name):
    # operators.py imports torch, which this package otherwise leaves to the first call
    if name in _OPERATORS:
        from . import operators
        globals().update({n: getattr(operators, n) for n in _OPERATORS})
        return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")


def __dir__():
    return sorted(set(globals()) | set(_OPERATORS))
