"""Expert products in 8-bit integers with a scale per row and per output channel:
Python binding of moe_int8_product (include/moe.h). The weights are the int8 arrays
and bf16 channel scales that the sublayer's int8-weight form takes.

One layer of any router, T tokens x [T, d], weights [E, d, f] and [E, f, d]:

    r = moe.moe_topk_route(logits, k)
    h = moe.moe_int8_product(x, w_gate, s_gate, index=r["perm_token"], counts=r["counts"],
                             w_up=w_up, s_up=s_up)
    y = moe.moe_int8_product(h, w_down, s_down, counts=r["counts"], gate=r["gate_perm"])
    out = moe.moe_combine_topk(y, r["slot_pos"])

Tensors, devices, streams and errors as in the routing calls.
"""

from __future__ import annotations

import ctypes

from . import _native as N
from .routed import _check, _codes, _need, _place, _refuse

__all__ = ["moe_int8_product", "moe_int8_workspace_size"]


def moe_int8_workspace_size(R, K, N_cols, n_experts=1, x_dtype=N.MOE_BF16, with_up=False) -> int:
    """Workspace bytes of moe_int8_product (0 on bad sizes or R == 0)."""
    return N.lib().moe_int8_workspace_size(R, K, N_cols, n_experts, x_dtype, int(bool(with_up)))


def moe_int8_product(x, w, s, *, x_scale=None, index=None, counts=None, w_up=None, s_up=None,
                     activation=N.MOE_ACT_GELU_TANH, gate=None, out=None, out_dtype=None, workspace=None, stream=None):
    """out[r] = gate[r] * (row r . w[e]) * s[e] for the rows r of expert e, or with
    ``w_up`` / ``s_up`` gate[r] * act(row . w[e] * s[e]) * (row . w_up[e] * s_up[e]).

    ``x`` [x_rows, K] in bf16 or fp32 is quantised on the way, row by row, ``index`` [R]
    (int32) choosing its rows; in int8 it is [R, K] with ``x_scale`` [R]. ``w`` [n, K, N]
    int8, ``s`` [n, N] bf16. ``counts`` [n] (int32, on the device): rows of each expert, in
    order; without it n must be 1. Rows of ``out`` [R, N] behind the last expert's are left
    as they were (an output that is not given starts as zeros then). ``out_dtype``: bf16
    (the default) or fp32. ``workspace``: uint8 tensor of moe_int8_workspace_size bytes;
    moe_device_status reads its status word."""
    import torch

    if x.dim() != 2 or w.dim() != 3:
        _refuse("x must be [rows, K] and w [n_experts, K, N]")
    n, K, cols = w.shape
    dev = x.device
    i8, b16 = torch.int8, torch.bfloat16
    x_code = N.MOE_INT8 if x.dtype == i8 else _codes().get(x.dtype)
    if x_code is None:
        _refuse(f"x has type {x.dtype}, not bf16, fp32 or int8")
    R = x.shape[0] if index is None else index.shape[0]
    if (w_up is None) != (s_up is None):
        _refuse("w_up and s_up come together")
    a = N.MoeInt8Args(
        _need(x, "x", (x.shape[0], K), (x.dtype,), None), _need(x_scale, "x_scale", (R,), (torch.float32,), dev),
        _need(index, "index", (R,), (torch.int32,), dev), _need(counts, "counts", (n,), (torch.int32,), dev),
        _need(w, "w", (n, K, cols), (i8,), dev), _need(w_up, "w_up", (n, K, cols), (i8,), dev),
        _need(s, "s", (n, cols), (b16,), dev), _need(s_up, "s_up", (n, cols), (b16,), dev),
        _need(gate, "gate", (R,), (torch.float32,), dev), None, x.shape[0], R, K, cols, n, x_code, N.MOE_BF16, activation)
    with _place(dev, stream) as handle:
        if out is None:
            out = (torch.empty if counts is None else torch.zeros)((R, cols), dtype=out_dtype or b16, device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            _refuse(f"out has type {out.dtype}, not {out_dtype}")
        a.out = _need(out, "out", (R, cols), (b16, torch.float32), dev)
        a.out_dtype = _codes()[out.dtype]
        if workspace is None:
            size = N.lib().moe_int8_workspace_size(R, K, cols, n, x_code, int(w_up is not None))
            workspace = torch.empty(size, dtype=torch.uint8, device=dev)
        st = N.lib().moe_int8_product(ctypes.byref(a), _need(workspace, "workspace", workspace.shape, (torch.uint8,), dev),
                                      workspace.numel(), handle)
    _check(st, "moe_int8_product")
    return out
