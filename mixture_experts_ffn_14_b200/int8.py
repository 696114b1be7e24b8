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

from . import _native as N
from . import routed as _r
from .routed import _check, _code, _first, _need, _on, _refuse

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
    dev = _first(x, "x", 2)
    _first(w, "w", 3)
    f32, i32, i8, b16 = _r._F32, _r._I32, _r._I8, _r._BF16
    rows, xt = x.shape[0], x.dtype
    n, K, cols = shape = w.shape
    x_code = N.MOE_INT8 if xt is i8 else _code(xt, "x")
    if x.shape[1] != K:
        _refuse(f"x has rows of {x.shape[1]}, w of {K}")
    R = rows if index is None else index.numel()
    if (w_up is None) != (s_up is None):
        _refuse("w_up and s_up come together")
    xp = x.data_ptr()
    ptrs = (_need(x_scale, "x_scale", (R,), f32, dev), _need(index, "index", (R,), i32, dev),
            _need(counts, "counts", (n,), i32, dev), _need(w, "w", shape, i8, dev),
            _need(w_up, "w_up", shape, i8, dev), _need(s, "s", (n, cols), b16, dev),
            _need(s_up, "s_up", (n, cols), b16, dev), _need(gate, "gate", (R,), f32, dev))

    def call(handle):
        o = out
        if o is None:
            import torch

            o = (torch.empty if counts is None else torch.zeros)((R, cols), dtype=out_dtype or b16, device=dev)
        elif out_dtype is not None and o.dtype is not out_dtype:
            _refuse(f"out has type {o.dtype}, not {out_dtype}")
        dtype = o.dtype
        out_code = _code(dtype, "out")
        a = N.MoeInt8Args(xp, *ptrs, _need(o, "out", (R, cols), dtype, dev), rows, R, K, cols, n, x_code, out_code,
                          activation)
        L = N.lib()
        if workspace is None:
            from torch import empty

            size = L.moe_int8_workspace_size(R, K, cols, n, x_code, 0 if w_up is None else 1)
            held = empty(size, dtype=_r._U8, device=dev)
            ws = held.data_ptr()
        else:
            size = workspace.numel()
            ws = _need(workspace, "workspace", (size,), _r._U8, dev)
        _check(L.moe_int8_product(a, ws, size, handle), "moe_int8_product")
        return o

    return _on(dev, stream, call)
