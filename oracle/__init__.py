"""Test infrastructure: the float64 CPU oracle for FAVOR+ attention, the selective scan, the short
causal convolution and the page calls.

Only the tests, ``__graft_entry__.smoke()`` and the CPU-baseline leg of
``bench.py`` may import this package.  The CUDA library never calls it and
shares no code with it.
"""
from .favor64 import *  # noqa: F401,F403
from .ssm64 import *  # noqa: F401,F403
from . import favor64 as _favor64, ssm64 as _ssm64

__all__ = _favor64.__all__ + _ssm64.__all__
