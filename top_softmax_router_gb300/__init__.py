"""Chunk-bounded, top-k-softmax-routed MoE block on one GB300 (sm_103a).

The compute lives in libmoe.so (hand-written CUDA; C ABI in include/moe*.h); this package is the build script and a thin ctypes binding.
"""
from .api import *  # noqa: F401,F403
from .adamw import *  # noqa: F401,F403
from .ce import *  # noqa: F401,F403
from .norm import *  # noqa: F401,F403
from .blocks8 import *  # noqa: F401,F403
from .rmsnorm import *  # noqa: F401,F403
from .linear import *  # noqa: F401,F403
from .embed import *  # noqa: F401,F403
from .scores import *  # noqa: F401,F403
from .distill import *  # noqa: F401,F403
from .autograd import *  # noqa: F401,F403
