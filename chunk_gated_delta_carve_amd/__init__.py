"""MI355X-native CARVE chunk-parallel layer (HIP kernels for gfx950 behind a C ABI): forward
pass, backward pass and decode step, and the operators of the attention layer that stands
beside it in a hybrid model: norm and rotation of queries and keys, a paged cache in bf16,
fp32 or 4 bits and attention over it, and the pages of the next tokens.

`chunk_fwd`, `chunk_bwd`, `recurrent_step`, `recurrent_ref_shapes` and the attention layer's
functions are imported lazily so that the input
generator (`workloads`) and the build script work without torch or the
compiled library.
"""

_ATTENTION = ("qk_norm_rope_fwd", "qk_norm_rope_bwd", "paged_append", "paged_attention", "paged_workspace_bytes",
              "rope_tables")
_FP4 = ("paged_assign", "paged_append_fp4", "paged_read_fp4", "paged_attention_fp4", "paged_fp4_cache",
        "paged_fp4_workspace_bytes")
__all__ = ["chunk_fwd", "chunk_bwd", "recurrent_step", "recurrent_ref_shapes", *_ATTENTION, *_FP4]


def __getattr__(name):
    if name in __all__:
        from . import api, attention, fp4
        value = getattr(attention if name in _ATTENTION else fp4 if name in _FP4 else api, name)
        globals()[name] = value
        return value
    raise AttributeError(name)
