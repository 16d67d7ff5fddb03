"""Binding of the grouped router, the grouping without copied rows, the 8-bit
quantiser, the block-scaled 8-bit products and the layer built of them.

Argument checks and marshalling only (include/moe.h says what each entry point
computes). 8-bit tensors are torch.float8_e4m3fn with torch.uint8 scales, one
E8M0 byte b (2^(b - 127)) for each block of 128 columns of a row (activations)
or of 128 x 128 (weights); a weight argument is the pair (values, scales).
"""
from __future__ import annotations

import ctypes
from typing import Dict, Optional, Tuple

import torch

from .binding import GemmFp8Desc, MoeDesc, RouterDesc, _check, lib
from . import workloads as W

_F8 = torch.float8_e4m3fn
_DTYPES = {torch.float32: W.DT_F32, torch.bfloat16: W.DT_BF16}
_SCORES = {"softmax": 0, "sigmoid": 1}
BLOCK = 128

Weight = Tuple[torch.Tensor, torch.Tensor]


# These calls run for microseconds on the GPU, so what they cost on the host counts: the raw stream and device queries
# take 0.1 and 0.2 us, where torch.cuda.current_stream() takes 3.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", lambda dev: torch.cuda.current_stream(dev).cuda_stream)
_device = torch.cuda.current_device


def _blocks(n: int) -> int:
    return (n + BLOCK - 1) // BLOCK


def _dtype(name: str, t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise ValueError("%s must be float32 or bfloat16, not %s" % (name, t.dtype))
    return _DTYPES[t.dtype]


def _arg(name: str, t: Optional[torch.Tensor], shape, dtype, device: int) -> Optional[int]:
    """Address of a contiguous tensor of this shape and type on the current device (None: not given)."""
    if t is None:
        return None
    if not t.is_cuda or t.get_device() != device:
        raise ValueError("%s must be on the current GPU (cuda:%d), not on %s" % (name, device, t.device))
    if t.shape != shape or t.dtype != dtype:
        raise ValueError("%s must be %s of shape %s, not %s of shape %s"
                         % (name, dtype, tuple(shape), t.dtype, tuple(t.shape)))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    return t.data_ptr() or None


def _weight(name: str, w: Optional[Weight], E: int, rows: int, cols: int, device: int):
    if w is None:
        return None, None
    return (_arg(name, w[0], (E, rows, cols), _F8, device),
            _arg(name + "'s scales", w[1], (E, _blocks(rows), _blocks(cols)), torch.uint8, device))


def _space(ws: torch.Tensor, device: int) -> Tuple[Optional[int], int]:
    if not ws.is_cuda or ws.get_device() != device or ws.dtype != torch.uint8 or not ws.is_contiguous():
        raise ValueError("the workspace must be a contiguous uint8 tensor on the current GPU")
    return ws.data_ptr() or None, ws.numel()


def router_desc(T: int, E: int, K: int, score: str = "softmax", renorm: bool = True, scale: float = 1.0,
                groups: int = 1, top_groups: Optional[int] = None, group_top: int = 1) -> RouterDesc:
    """A router over T tokens and E experts (moe_router_desc): `score` is "softmax" or "sigmoid"; with groups > 1 only
    the top_groups best groups (by the sum of their group_top best experts) can be chosen from; gates are the chosen
    scores, renormalised to sum to 1 unless renorm is False, times scale."""
    if score not in _SCORES:
        raise ValueError("score must be 'softmax' or 'sigmoid', not %r" % (score,))
    return RouterDesc(T, E, K, groups, groups if top_groups is None else top_groups, group_top, _SCORES[score],
                      1 if renorm else 0, scale)


def route_grouped(desc: RouterDesc, logits: torch.Tensor, bias: Optional[torch.Tensor] = None,
                  topk_idx: Optional[torch.Tensor] = None,
                  topk_gate: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_route_grouped: choice and gates for logits [T][E] (float32 or bfloat16); bias [E] float32 steers the choice
    only. Returns topk_idx [T][K] int32 and topk_gate [T][K] float32 (written in place if given)."""
    dev = _device()
    T, E, K = desc.T, desc.E, desc.K
    topk_idx = logits.new_empty((T, K), dtype=torch.int32) if topk_idx is None else topk_idx
    topk_gate = logits.new_empty((T, K), dtype=torch.float32) if topk_gate is None else topk_gate
    _check("moe_route_grouped", lib().moe_route_grouped(
        ctypes.byref(desc), _arg("logits", logits, (T, E), logits.dtype, dev), _dtype("logits", logits),
        _arg("bias", bias, (E,), torch.float32, dev), _arg("topk_idx", topk_idx, (T, K), torch.int32, dev),
        _arg("topk_gate", topk_gate, (T, K), torch.float32, dev), _raw_stream(dev)))
    return {"topk_idx": topk_idx, "topk_gate": topk_gate}


def route_grouped_backward(desc: RouterDesc, logits: torch.Tensor, topk_idx: torch.Tensor, dgate: torch.Tensor,
                           dlogits: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_route_grouped_backward: the gradient of sum(dgate * topk_gate) with respect to the logits, in their type."""
    dev = _device()
    T, E, K = desc.T, desc.E, desc.K
    dlogits = torch.empty_like(logits) if dlogits is None else dlogits
    _check("moe_route_grouped_backward", lib().moe_route_grouped_backward(
        ctypes.byref(desc), _arg("logits", logits, (T, E), logits.dtype, dev), _dtype("logits", logits),
        _arg("topk_idx", topk_idx, (T, K), torch.int32, dev), _arg("dgate", dgate, (T, K), torch.float32, dev),
        _arg("dlogits", dlogits, (T, E), logits.dtype, dev), _raw_stream(dev)))
    return dlogits


def group_workspace(T: int, E: int, K: int, device="cuda") -> torch.Tensor:
    """A workspace for group() of T tokens' K choices over E experts."""
    n = ctypes.c_size_t(0)
    _check("moe_group_workspace_size", lib().moe_group_workspace_size(T, E, K, ctypes.byref(n)))
    return torch.empty(max(n.value, 256), dtype=torch.uint8, device=device)


def group(topk_idx: torch.Tensor, E: int, ws: Optional[torch.Tensor] = None) -> Dict[str, torch.Tensor]:
    """moe_group: stable grouping of the choices topk_idx [T][K] by expert: counts [E], offsets [E+1], slot_token [T*K],
    token_slot [T][K] (all int32)."""
    dev = _device()
    if topk_idx.dim() != 2 or topk_idx.dtype != torch.int32:
        raise ValueError("topk_idx must be [T][K] and int32")
    T, K = topk_idx.shape
    ws = group_workspace(T, E, K, topk_idx.device) if ws is None else ws
    # one allocation, each output on a multiple of 16 bytes
    S = T * K
    n, p = -E % 4, -S % 4
    buf = topk_idx.new_empty(2 * (E + S) + 1 + n + 2 * p)
    if n == 0 and p == 0:
        counts, slot_token, token_slot, offsets = buf.split_with_sizes((E, S, S, E + 1))
    else:
        counts, _, slot_token, _, token_slot, _, offsets = buf.split_with_sizes((E, n, S, p, S, p, E + 1))
    out = {"counts": counts, "offsets": offsets, "slot_token": slot_token, "token_slot": token_slot.view(T, K)}
    _check("moe_group", lib().moe_group(
        T, E, K, _arg("topk_idx", topk_idx, (T, K), torch.int32, dev), counts.data_ptr(),
        offsets.data_ptr(), slot_token.data_ptr() or None, token_slot.data_ptr() or None,
        *_space(ws, dev), _raw_stream(dev)))
    return out


def quantize_fp8(x: torch.Tensor, block_rows: int = 1) -> Weight:
    """moe_quantize_fp8: x [..., rows, cols] (float32 or bfloat16) to e4m3 values of the same shape and one E8M0 byte per
    block of block_rows (1 or 128) x 128: [..., ceil(rows / block_rows), ceil(cols / 128)]."""
    dev = _device()
    if x.dim() < 2:
        raise ValueError("x must have rows and columns")
    *lead, rows, cols = x.shape
    mats = 1
    for n in lead:
        mats *= n
    px = _arg("x", x, x.shape, x.dtype, dev)
    q = torch.empty_like(x, dtype=_F8)
    scale = x.new_empty((*lead, (rows + block_rows - 1) // max(block_rows, 1), (cols + BLOCK - 1) // BLOCK),
                        dtype=torch.uint8)
    _check("moe_quantize_fp8", lib().moe_quantize_fp8(px, _dtype("x", x), mats, rows, cols, block_rows,
                                                      q.data_ptr() or None, scale.data_ptr() or None, _raw_stream(dev)))
    return q, scale


def grouped_gemm_fp8(x: torch.Tensor, x_scale: torch.Tensor, weight: torch.Tensor, weight_scale: torch.Tensor,
                     offsets: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
                     bias: Optional[torch.Tensor] = None, max_rows: int = 0, out_dtype: torch.dtype = torch.bfloat16,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_grouped_gemm_fp8: out[s] = W_e x[rows[s]] (+ bias_e) for the grouped rows s of expert e. weight [E][N][Kd] (or
    [N][Kd]: one expert, offsets may be left out); rows [S] int32 (None: row s itself). out [S][N]; rows that no expert
    holds are left as they were."""
    dev = _device()
    if x.dim() != 2 or weight.dim() not in (2, 3):
        raise ValueError("x must be [rows][Kd] and the weight [E][N][Kd] or [N][Kd]")
    n, Kd = x.shape
    N = weight.shape[-2]
    E = weight.shape[0] if weight.dim() == 3 else 1
    lead = (E,) if weight.dim() == 3 else ()
    S = n if rows is None else rows.numel()
    if out is None:
        out = torch.empty((S, N), dtype=out_dtype, device=x.device)
    bt = 0 if bias is None else _dtype("bias", bias)
    desc = GemmFp8Desc(S, n, E, N, Kd, max_rows, _dtype("out", out), bt)
    _check("moe_grouped_gemm_fp8", lib().moe_grouped_gemm_fp8(
        ctypes.byref(desc), _arg("x", x, (n, Kd), _F8, dev),
        _arg("x_scale", x_scale, (n, _blocks(Kd)), torch.uint8, dev), _arg("rows", rows, (S,), torch.int32, dev),
        _arg("offsets", offsets, (E + 1,), torch.int32, dev), _arg("weight", weight, lead + (N, Kd), _F8, dev),
        _arg("weight_scale", weight_scale, lead + (_blocks(N), _blocks(Kd)), torch.uint8, dev),
        _arg("bias", bias, lead + (N,), None if bias is None else bias.dtype, dev),
        _arg("out", out, (S, N), out.dtype, dev), _raw_stream(dev)))
    return out


def fp8_workspace(desc: MoeDesc, device="cuda") -> torch.Tensor:
    """A workspace for expert_ffn_fp8 and forward_fp8."""
    n = ctypes.c_size_t(0)
    _check("moe_fp8_workspace_size", lib().moe_fp8_workspace_size(ctypes.byref(desc), ctypes.byref(n)))
    return torch.empty(max(n.value, 256), dtype=torch.uint8, device=device)


def _experts(desc: MoeDesc, W1: Weight, W3: Optional[Weight], W2: Weight, b1, b2, dev: int):
    E, d, w = desc.E, desc.d, desc.width
    dt = torch.bfloat16 if desc.dtype == W.DT_BF16 else torch.float32
    return (*_weight("W1", W1, E, w, d, dev), _arg("b1", b1, (E, w), dt, dev), *_weight("W3", W3, E, w, d, dev),
            *_weight("W2", W2, E, d, w, dev), _arg("b2", b2, (E, d), dt, dev))


def expert_ffn_fp8(desc: MoeDesc, x: torch.Tensor, x_scale: torch.Tensor, offsets: torch.Tensor, W1: Weight,
                   W3: Optional[Weight], W2: Weight, b1: Optional[torch.Tensor] = None,
                   b2: Optional[torch.Tensor] = None, rows: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None, o_perm: Optional[torch.Tensor] = None) -> torch.Tensor:
    """moe_expert_ffn_fp8: float32 ungated expert outputs [T*K][d] of the grouped rows x [T*K][d], or with
    rows = slot_token of the tokens' x [T][d]."""
    dev = _device()
    T, S, d = desc.T, desc.T * desc.K, desc.d
    n = S if rows is None else T
    ws = fp8_workspace(desc, x.device) if ws is None else ws
    o_perm = torch.empty((S, d), dtype=torch.float32, device=x.device) if o_perm is None else o_perm
    _check("moe_expert_ffn_fp8", lib().moe_expert_ffn_fp8(
        ctypes.byref(desc), _arg("x", x, (n, d), _F8, dev), _arg("x_scale", x_scale, (n, _blocks(d)), torch.uint8, dev),
        _arg("rows", rows, (S,), torch.int32, dev), _arg("offsets", offsets, (desc.E + 1,), torch.int32, dev),
        *_experts(desc, W1, W3, W2, b1, b2, dev), _arg("o_perm", o_perm, (S, d), torch.float32, dev),
        *_space(ws, dev), _raw_stream(dev)))
    return o_perm


def forward_fp8(desc: MoeDesc, router: RouterDesc, h: torch.Tensor, logits: torch.Tensor,
                bias: Optional[torch.Tensor], W1: Weight, W3: Optional[Weight], W2: Weight,
                b1: Optional[torch.Tensor] = None, b2: Optional[torch.Tensor] = None,
                ws: Optional[torch.Tensor] = None, y: Optional[torch.Tensor] = None,
                counts: Optional[torch.Tensor] = None, topk_idx: Optional[torch.Tensor] = None,
                topk_gate: Optional[torch.Tensor] = None) -> Tuple[torch.Tensor, torch.Tensor]:
    """moe_forward_fp8: the layer on given router logits [T][E] with 8-bit weights: (y, counts). topk_idx and topk_gate
    are written if given."""
    dev = _device()
    T, E, K, d = desc.T, desc.E, desc.K, desc.d
    dt = torch.bfloat16 if desc.dtype == W.DT_BF16 else torch.float32
    ws = fp8_workspace(desc, h.device) if ws is None else ws
    y = torch.empty((T, d), dtype=dt, device=h.device) if y is None else y
    counts = torch.empty(E, dtype=torch.int32, device=h.device) if counts is None else counts
    _check("moe_forward_fp8", lib().moe_forward_fp8(
        ctypes.byref(desc), ctypes.byref(router), _arg("h", h, (T, d), dt, dev),
        _arg("logits", logits, (T, E), logits.dtype, dev), _dtype("logits", logits),
        _arg("bias", bias, (E,), torch.float32, dev), *_experts(desc, W1, W3, W2, b1, b2, dev),
        _arg("y", y, (T, d), dt, dev), _arg("topk_idx", topk_idx, (T, K), torch.int32, dev),
        _arg("topk_gate", topk_gate, (T, K), torch.float32, dev), _arg("counts", counts, (E,), torch.int32, dev),
        *_space(ws, dev), _raw_stream(dev)))
    return y, counts
