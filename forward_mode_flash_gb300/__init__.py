"""GB300-native fused attention forward + JVP (forward-mode flash attention).

The compute lives in the CUDA library built from ``csrc/`` (see ``build.py``);
this package holds the ctypes binding (``attention``), work/traffic counts
(``metrics``) and the seeded input generators shared with the tests
(``synth``).  Importing the package does not load the library; the first call
does, and raises if it has not been built.
"""

from .api import (attention, attention_chunk, attention_decode, attention_packed,  # noqa: F401
                  cache_append, cache_read, cache_write, device_status, fwd_dual, last_path,
                  norm_rope, rope_table)

__all__ = ["attention", "attention_chunk", "attention_decode", "attention_packed", "cache_append",
           "cache_read", "cache_write", "fwd_dual", "device_status", "last_path", "norm_rope",
           "rope_table"]
