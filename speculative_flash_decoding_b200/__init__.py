"""Speculative flash-decode attention (attention-level speculation) for B200.

For every decode query the library computes, in CUDA kernels for sm_100a,
the attention-sink approximation O_spec (softmax attention over the first S
and last W cached tokens, published early by a kernel launched first at high
priority, with the exact path running beside it), the exact attention
O_exact over the whole cache (split-K flash decoding), the per-token
relative L2 error of O_spec and the commit/discard flag.

Beside it, what a decode layer over a paged cache needs: pages written
(quantised to e4m3 on request) and read back (``PagedCache``), attention of
one new token per sequence over its pages (``PagedDecoder``) and a linear
layer with its epilogue (``Linear``).

The C ABI is include/alspec.h (libalspec.so); ``alspec`` is its ctypes
binding.  Importing the package raises if libalspec.so is missing.  torch is
imported where its tensors are taken, not with the package: the binding needs
none.
"""
from importlib import import_module as _import_module
from importlib.util import find_spec as _find_spec

from .alspec import *  # noqa: F401,F403
from .alspec import Decoder, AlspecError, make_desc, SIGNATURES, LIB_PATH  # noqa: F401

__version__ = "0.1.0"

# What takes torch tensors, and its module.
_TENSOR_LAYER = {"Linear": ".linear", "PagedCache": ".paged", "PagedDecoder": ".paged",
                 "linear": ".linear", "paged": ".paged"}

# `import *` brings them where there is a torch.
__all__ = [name for name in dir() if not name.startswith("_")]
if _find_spec("torch"):
    __all__ += _TENSOR_LAYER


def __getattr__(name):
    if name not in _TENSOR_LAYER:
        raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
    module = _import_module(_TENSOR_LAYER[name], __name__)
    value = module if name.islower() else getattr(module, name)
    globals()[name] = value  # found there from now on
    return value


def __dir__():
    return sorted({*globals(), *_TENSOR_LAYER})
