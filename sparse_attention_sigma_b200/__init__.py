"""B200-native (sm_100a) inference forward pass of Hamming Attention Distillation.

The work happens in the CUDA library ``libhad.so`` behind the C ABI declared
in ``include/had.h``; ``had`` is its thin ctypes binding, and ``cache`` that
of the decoder cache.  Importing the package does not load the library;
``from sparse_attention_sigma_b200 import had`` (or ``cache``) does, and
fails loudly if it is missing.
"""
import importlib

__all__ = ["had", "cache"]


def __getattr__(name):
    if name in __all__:
        return importlib.import_module(__name__ + "." + name)
    raise AttributeError(name)
