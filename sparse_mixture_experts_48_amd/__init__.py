"""Top-K routed mixture-of-experts FFN layer (forward pass) for the AMD MI355X.

The compute lives in libmoe_mi355x.so (hand-written HIP for gfx950, C-ABI in
include/moe.h); this package holds its ctypes binding, the build script and the
seeded synthetic workloads.
"""
from . import workloads  # noqa: F401
from .binding import (GemmFp8Desc, MoeDesc, MoeError, MoELayer, RouterDesc, Trace, backward, backward_workspace, capacity_slots,  # noqa: F401
                      combine, desc_of, expert_ffn, forward, forward_noalloc, header_symbols, lib, permute, route,
                      workspace, workspace_size)
from .fp8 import (expert_ffn_fp8, forward_fp8, fp8_workspace, group, group_workspace, grouped_gemm_fp8,  # noqa: F401
                  quantize_fp8, route_grouped, route_grouped_backward, router_desc)
