"""GB300 (sm_103a) NVFP4 W4A16 block-scaled linear layer.

The compute lives in ``libnvfp4_linear.so`` (CUDA, built from ``csrc/``);
``linear``, ``linear_swiglu`` and friends are thin ctypes marshalling around
its C ABI (``include/nvfp4_linear.h``).  The attention block's operators
between the projections (``include/nvfp4_attention.h``, ``csrc_attention/``)
are bound in ``attention``, those of layers whose activations are NVFP4 too
(``include/nvfp4_w4a4.h``, ``csrc_w4a4/``) in ``w4a4``.  Nothing here computes on the CPU: if the library
or a GPU is missing, every call raises.
"""
import importlib

from .inputs import WORKLOADS, LinearInputs, algorithmic_bytes, flops  # noqa: F401


# The attention block's names (of the module ``attention``).
_ATTENTION = frozenset((
    "KVCache", "new_kv_cache", "qk_norm_rope", "qk_norm_rope_store", "attention_workspace",
    "release_workspaces", "paged_attention", "attention_mass", "evict", "attention_error", "ATTENTION_TIMEOUT",
    "ATTENTION_BAD_INDEX"))

# The NVFP4 x NVFP4 operators' names (of the module ``w4a4``).
_W4A4 = frozenset((
    "Fp4Rows", "new_fp4_rows", "Fp4Weight", "quantize_rows", "add_rms_norm", "add_rms_norm_quantize",
    "linear_w4a4", "linear_w4a4_swiglu", "linear_w4a4_swiglu_quantize", "w4a4_error", "W4A4_TIMEOUT"))


def __getattr__(name):
    # The bindings (every public name of _lib: the calls, the flag and kernel
    # constants; the attention block's and the NVFP4 x NVFP4 operators) are
    # imported lazily so that the input generators stay importable on machines
    # without the built library.  The operators' names are kept here once looked up:
    # finding one anew takes as long as a third of a call.
    for names, module in ((_ATTENTION, ".attention"), (_W4A4, ".w4a4")):
        if name in names:
            found = globals()[name] = getattr(importlib.import_module(module, __name__), name)
            return found
    if not name.startswith("_"):
        from . import _lib
        if hasattr(_lib, name):
            return getattr(_lib, name)
    raise AttributeError(name)
