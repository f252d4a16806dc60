"""FAVOR+ attention (Performers) and the selective state space scan for one GB300: a C-ABI CUDA
library (libfavor.so, kernels for sm_103a) and its ctypes binding."""
from . import favor as _favor, ssm as _ssm
from .favor import *  # noqa: F401,F403
from .ssm import *  # noqa: F401,F403

__all__ = _favor.__all__ + _ssm.__all__
