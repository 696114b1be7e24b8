"""Routing, its gradient and the combine of any number of experts and choices
per token: Python binding of the C calls of the same names (include/moe.h).

Every tensor is dense, on one CUDA device, which need not be the current one;
the work goes to ``stream`` (a torch stream or a handle), by default that
device's current stream. Outputs and workspaces that are not given are allocated
on that stream. Wrong shapes, types and devices raise ``ValueError``, a call that
the library refuses ``MoeError``; nothing is launched in either case.

    r = moe.moe_topk_route(logits, 8, score=moe.MOE_SCORE_SIGMOID, bias=bias, renormalize=True)
    ...                                  # experts on rows r["perm_token"], gates r["gate_perm"]
    out = moe.moe_combine_topk(y, r["slot_pos"])
"""

from __future__ import annotations

import contextlib
import ctypes

from . import _native as N

__all__ = ["moe_topk_route", "moe_topk_route_backward", "moe_topk_workspace_size", "moe_combine_topk"]

_CODES = None


def _codes():
    """dtype codes of the types the calls take."""
    global _CODES
    if _CODES is None:
        import torch

        _CODES = {torch.float32: N.MOE_F32, torch.bfloat16: N.MOE_BF16}
    return _CODES


def _refuse(what):
    raise ValueError("moe: " + what)


def _need(t, name, shape, dtypes, device):
    """Check one tensor; returns its address (None for an absent one)."""
    if t is None:
        return None
    if not t.is_cuda:
        _refuse(f"{name} must live on a CUDA device")
    if device is not None and t.device != device:
        _refuse(f"{name} is on {t.device}, the call's other tensors on {device}")
    if t.dtype not in dtypes:
        _refuse(f"{name} has type {t.dtype}, not {' or '.join(str(d) for d in dtypes)}")
    if tuple(t.shape) != tuple(shape):
        _refuse(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
    if not t.is_contiguous():
        _refuse(f"{name} must be contiguous")
    return t.data_ptr()


@contextlib.contextmanager
def _place(device, stream):
    """Make `device` current, and `stream` with it if one is given (so that what is
    allocated inside belongs to it); yields the stream's handle."""
    import torch

    with torch.cuda.device(device):
        if stream is None:
            yield torch.cuda.current_stream(device).cuda_stream
            return
        s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
        if s.device != device:
            _refuse(f"stream is on {s.device}, the tensors on {device}")
        with torch.cuda.stream(s):
            yield s.cuda_stream


def _check(status, what):
    if status != N.MOE_OK:
        from . import MoeError

        raise MoeError(status, what)


def moe_topk_workspace_size(T, E, k) -> int:
    """Workspace bytes of moe_topk_route with the dispatch (0: none needed)."""
    return N.lib().moe_topk_workspace_size(T, E, k)


def _topk_args(logits, k, score, n_groups, topk_groups, group_rule, renormalize, scale, bias, n_tokens):
    import torch

    if logits.dim() != 2:
        _refuse("logits must be [T, E]")
    T, E = logits.shape
    dev = logits.device
    a = N.MoeTopkArgs(_need(logits, "logits", (T, E), (torch.float32, torch.bfloat16), None),
                      _need(bias, "bias", (E,), (torch.float32,), dev),
                      None, T, E, k, _codes()[logits.dtype], score, n_groups, topk_groups, group_rule,
                      int(bool(renormalize)), float(scale))
    if n_tokens is not None:
        if n_tokens.numel() != 1:
            _refuse("n_tokens must hold one number")
        a.n_tokens = _need(n_tokens, "n_tokens", n_tokens.shape, (torch.int32,), dev)
    return a


_DISPATCH = ("counts", "offsets", "perm_token", "perm_slot", "slot_pos", "gate_perm")


def moe_topk_route(logits, k, *, score=N.MOE_SCORE_SOFTMAX, bias=None, n_groups=1, topk_groups=1,
                   group_rule=N.MOE_GROUP_MAX, renormalize=False, scale=1.0, n_tokens=None, want_scores=False,
                   dispatch=True, out=None, workspace=None, stream=None) -> dict:
    """Route logits [T, E] (fp32 or bf16) to k experts per token. Returns a dict with
    ``idx`` [T, k] (int32, -1 = none), ``weights`` [T, k], ``scores`` [T, E] if
    ``want_scores``, and with ``dispatch`` the stable (expert, token) order of the
    choice: ``counts`` [E], ``offsets`` [E+1], ``perm_token`` and ``perm_slot`` [T*k],
    ``slot_pos`` [T, k], ``gate_perm`` [T*k]. ``n_tokens``: a one-element int32 tensor,
    rows from it on are padding. ``out``: a dict of such tensors to write into (those it
    lacks are allocated). ``workspace``: uint8 tensor of moe_topk_workspace_size bytes."""
    import torch

    a = _topk_args(logits, k, score, n_groups, topk_groups, group_rule, renormalize, scale, bias, n_tokens)
    T, E, dev = a.T, a.E, logits.device
    n = max(0, k)
    shapes = {"idx": ((T, n), torch.int32), "weights": ((T, n), torch.float32)}
    if want_scores:
        shapes["scores"] = ((T, E), torch.float32)
    if dispatch:
        shapes.update(counts=((E,), torch.int32), offsets=((E + 1,), torch.int32),
                      perm_token=((T * n,), torch.int32), perm_slot=((T * n,), torch.int32),
                      slot_pos=((T, n), torch.int32), gate_perm=((T * n,), torch.float32))
    given = out or {}
    if unknown := set(given) - set(shapes):
        _refuse(f"out holds {sorted(unknown)}, which this call does not write")
    with _place(dev, stream) as handle:
        res = {}
        r = N.MoeTopkRouted()
        for name, (shape, dtype) in shapes.items():
            t = given.get(name)
            if t is None:
                t = torch.empty(shape, dtype=dtype, device=dev)
            res[name] = t
            setattr(r, name, _need(t, name, shape, (dtype,), dev))
        need = N.lib().moe_topk_workspace_size(T, E, n) if dispatch else 0
        if workspace is None and need:
            workspace = torch.empty(need, dtype=torch.uint8, device=dev)
        ws = _need(workspace, "workspace", (workspace.numel(),), (torch.uint8,), dev) if workspace is not None else None
        st = N.lib().moe_topk_route(ctypes.byref(a), ctypes.byref(r), ws, workspace.numel() if ws else 0, handle)
    _check(st, "moe_topk_route")
    return res


def moe_topk_route_backward(logits, idx, grad_weights, *, score=N.MOE_SCORE_SOFTMAX, renormalize=False, scale=1.0,
                            grad_scores=None, n_tokens=None, out=None, stream=None):
    """Gradient of moe_topk_route's ``weights`` (and ``scores``, if ``grad_scores`` [T, E]
    is given) to the logits, in the logits' type, for its choice ``idx``."""
    import torch

    if idx.dim() != 2:
        _refuse("idx must be [T, k]")
    k = idx.shape[1]
    a = _topk_args(logits, k, score, 1, 1, N.MOE_GROUP_MAX, renormalize, scale, None, n_tokens)
    dev = logits.device
    with _place(dev, stream) as handle:
        if out is None:
            out = torch.empty_like(logits)
        st = N.lib().moe_topk_route_backward(
            ctypes.byref(a), _need(idx, "idx", (a.T, k), (torch.int32,), dev),
            _need(grad_weights, "grad_weights", (a.T, k), (torch.float32,), dev),
            _need(grad_scores, "grad_scores", (a.T, a.E), (torch.float32,), dev),
            _need(out, "out", (a.T, a.E), (logits.dtype,), dev), handle)
    _check(st, "moe_topk_route_backward")
    return out


def moe_combine_topk(y, slot_pos, *, weights=None, residual=None, out=None, out_dtype=None, stream=None):
    """out[t] = residual[t] + sum_s weights[t, s] * y[slot_pos[t, s]] for rows y [R, d]
    and slot_pos [T, k] (int32; entries outside [0, R) add nothing). The output has
    ``out_dtype`` (bf16 or fp32), by default the residual's type, else y's."""
    import torch

    if y.dim() != 2 or slot_pos.dim() != 2:
        _refuse("y must be [R, d] and slot_pos [T, k]")
    (R, d), (T, k) = y.shape, slot_pos.shape
    dev, both = y.device, (torch.float32, torch.bfloat16)
    yp = _need(y, "y", (R, d), both, None)
    with _place(dev, stream) as handle:
        if out is None:
            out = torch.empty((T, d), dtype=out_dtype or (y.dtype if residual is None else residual.dtype), device=dev)
        elif out_dtype is not None and out.dtype != out_dtype:
            _refuse(f"out has type {out.dtype}, not {out_dtype}")
        op = _need(out, "out", (T, d), both, dev)
        st = N.lib().moe_combine_topk(yp, _codes()[y.dtype], R, _need(slot_pos, "slot_pos", (T, k), (torch.int32,), dev),
                                      _need(weights, "weights", (T, k), (torch.float32,), dev), T, k, d,
                                      _need(residual, "residual", (T, d), (out.dtype,), dev), op,
                                      _codes()[out.dtype], handle)
    _check(st, "moe_combine_topk")
    return out
