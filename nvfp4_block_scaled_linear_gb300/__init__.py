"""GB300 (sm_103a) NVFP4 W4A16 block-scaled linear layer.

The compute lives in ``libnvfp4_linear.so`` (CUDA, built from ``csrc/``);
``linear``, ``linear_swiglu`` and friends are thin ctypes marshalling around
its C ABI (``include/nvfp4_linear.h``).  The attention block's operators
between the projections (``include/nvfp4_attention.h``, ``csrc_attention/``)
are bound in ``attention``.  Nothing here computes on the CPU: if the library
or a GPU is missing, every call raises.
"""
import importlib

from .inputs import WORKLOADS, LinearInputs, algorithmic_bytes, flops  # noqa: F401


# The attention block's names (of the module ``attention``).
_ATTENTION = frozenset((
    "KVCache", "new_kv_cache", "qk_norm_rope", "qk_norm_rope_store", "attention_workspace",
    "release_workspaces", "paged_attention", "attention_mass", "evict", "attention_error", "ATTENTION_TIMEOUT",
    "ATTENTION_BAD_INDEX"))


def __getattr__(name):
    # The bindings (every public name of _lib: the calls, the flag and kernel
    # constants; the attention block's operators) are imported lazily so that
    # the input generators stay importable on machines without the built
    # library.
    if name in _ATTENTION:
        return getattr(importlib.import_module(".attention", __name__), name)
    if not name.startswith("_"):
        from . import _lib
        if hasattr(_lib, name):
            return getattr(_lib, name)
    raise AttributeError(name)
