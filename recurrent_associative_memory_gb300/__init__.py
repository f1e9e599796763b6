"""GB300-native generalised gated delta-rule recurrence (GDN, KLA, PGDN, Diagonal KDN).

The compute lives in ``libdr.so`` (CUDA for sm_103a behind the C ABI of
include/dr.h).  ``dr`` is its ctypes binding, ``runner`` allocates outputs and
calls it, ``workloads`` draws the seeded synthetic inputs, ``build`` compiles
the library.  ``attention`` (sliding window with sinks) and ``ssm`` (short
causal convolution, selective scan) are the layers that stand next to the
recurrence in a hybrid stack, and ``hybrid`` is such a stack.  Importing ``dr``
(or what calls it) requires the built library.
"""

__all__ = ["workloads", "build"]
