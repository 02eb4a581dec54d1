"""qstate for MI355X: decode step of gated linear recurrences with a low-bit state.

The compute path is libqstate.so (hand-written gfx950 kernels behind the C
ABI in include/qstate.h); this package holds the kernels' sources, the
build step, a ctypes binding and the seeded workload generators.  Besides
the step there is what a server needs around it: the scan of a prompt into a
state (QState.scan), the short causal convolution and the norm and rotation
of queries and keys before it, and copies of state slots (QState.copy_slots,
QState.compact_slots).
Importing the package loads nothing; the library is loaded on first use.
"""
from .api import QState, StateConfig, build_map, plan  # noqa: F401
from .ops import causal_conv, causal_conv_step, qk_norm_rotate  # noqa: F401

__all__ = ["QState", "StateConfig", "build_map", "plan", "causal_conv", "causal_conv_step", "qk_norm_rotate"]
