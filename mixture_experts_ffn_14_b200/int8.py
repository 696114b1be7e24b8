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
    moe_device_status reads its status word (bit 0x40: counts that are negative or run past
    the rows were cut off)."""
    call = (_r._calls or _r._load()).int8_product
    args = (x, w, s, x_scale, index, counts, w_up, s_up, activation, gate, out, out_dtype, workspace)
    return call(*args) if stream is None else _r._on(stream, x, call, args)
