"""B200-native fused decode FFN half-layer ("mono" kernel) and the attention
half's decode operators: a C-ABI CUDA library (libmonoffn.so, include/mono_ffn.h
and include/mono_attn.h) and its thin Python binding."""

from .binding import Plan, MonoError, lib  # noqa: F401

_ATTN = ("Rope", "rope", "KVCache", "AttnPlan", "Projection")


def __getattr__(name):   # attn.py imports torch; binding.py does so only where it needs it
    if name in _ATTN:
        from . import attn
        value = globals()[name] = getattr(attn, name)
        return value
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
