"""MI355X-native routed-MoE layer served from a per-layer GPU cache of hot experts.

The work happens in libmoecache.so (HIP kernels for gfx950 plus a C++ host
runtime) behind the C ABI of include/moe_cache.h; `binding` marshals arguments
to it with ctypes.  `decoder` holds the operators of the decoder layer around
the MoE layer, `step` those between a prompt and its next token (torch tensors).
Build the library with `python -m expert_cache_host_amd.build`.
"""
from .binding import (MISS_HOST, MISS_STREAM, MoECache, MoeError, Planner,  # noqa: F401
                      host_expert_forward, host_topk, lib_path, load_library, slot_bytes)


# by the module that holds them
_TORCH_OPS = {"decoder": ("KVCache", "Q4Matrix", "block_norm", "q4_matvec"),
              "step": ("Q8Matrix", "Q8Rows", "RoutingRule", "q8_matmul", "q8_rows", "route_experts", "sample_tokens")}


def __getattr__(name):
    # these operators take torch tensors: torch is imported with them
    for module, names in _TORCH_OPS.items():
        if name in names:
            import importlib
            ops = importlib.import_module("." + module, __name__)
            globals().update({n: getattr(ops, n) for n in names})
            return globals()[name]
    raise AttributeError(f"module {__name__!r} has no attribute {name!r}")
