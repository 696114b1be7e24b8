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

from . import _native as N

__all__ = ["moe_topk_route", "moe_topk_route_backward", "moe_topk_workspace_size", "moe_combine_topk"]

_CODES = {}
_F32 = _BF16 = _I32 = _I8 = _U8 = None
_current_device = _raw_stream = None


def _setup():
    """The torch names the calls use, looked up once (the package imports without torch)."""
    global _F32, _BF16, _I32, _I8, _U8, _current_device, _raw_stream
    import torch

    _F32, _BF16, _I32, _I8, _U8 = torch.float32, torch.bfloat16, torch.int32, torch.int8, torch.uint8
    _current_device = torch.cuda.current_device
    # the handle of a device's current stream without building a stream object for it
    _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
        lambda index: torch.cuda.current_stream(index).cuda_stream)
    _CODES.update({_F32: N.MOE_F32, _BF16: N.MOE_BF16})  # last: it says that the rest is there


def _refuse(what):
    raise ValueError("moe: " + what)


def _first(t, name, dims):
    """Check the tensor that the others are held against; returns its device."""
    if not _CODES:
        _setup()
    if not t.is_cuda:
        _refuse(f"{name} must live on a CUDA device")
    if t.dim() != dims:
        _refuse(f"{name} must have {dims} dimensions, not {t.dim()}")
    if not t.is_contiguous():
        _refuse(f"{name} must be contiguous")
    return t.device


def _need(t, name, shape, dtype, device):
    """Check one tensor; returns its address (None for an absent one)."""
    if t is None:
        return None
    if t.dtype is not dtype or t.shape != shape or t.device != device or not t.is_contiguous():
        if t.device != device:
            _refuse(f"{name} is on {t.device}, the call's other tensors on {device}")
        if t.dtype is not dtype:
            _refuse(f"{name} has type {t.dtype}, not {dtype}")
        if t.shape != shape:
            _refuse(f"{name} has shape {tuple(t.shape)}, not {tuple(shape)}")
        _refuse(f"{name} must be contiguous")
    return t.data_ptr()


def _code(dtype, name):
    code = _CODES.get(dtype)
    if code is None:
        _refuse(f"{name} has type {dtype}, not fp32 or bf16")
    return code


def _on(device, stream, call):
    """Run call(stream handle) with `device` current, and `stream` with it if one is given
    (so that what the call allocates belongs to that stream)."""
    if stream is None and _current_device() == device.index:
        return call(_raw_stream(device.index))
    import torch

    with torch.cuda.device(device):
        if stream is None:
            return call(_raw_stream(device.index))
        s = torch.cuda.ExternalStream(stream, device=device) if isinstance(stream, int) else stream
        if s.device != device:
            _refuse(f"stream is on {s.device}, the tensors on {device}")
        with torch.cuda.stream(s):
            return call(s.cuda_stream)


def _check(status, what):
    if status != N.MOE_OK:
        from . import MoeError

        raise MoeError(status, what)


def moe_topk_workspace_size(T, E, k) -> int:
    """Workspace bytes of moe_topk_route with the dispatch (0: none needed)."""
    return N.lib().moe_topk_workspace_size(T, E, k)


def _topk_args(logits, dev, k, score, n_groups, topk_groups, group_rule, renormalize, scale, bias, n_tokens):
    T, E = logits.shape
    nt = None
    if n_tokens is not None:
        if n_tokens.numel() != 1:
            _refuse("n_tokens must hold one number")
        nt = _need(n_tokens, "n_tokens", n_tokens.shape, _I32, dev)
    return N.MoeTopkArgs(logits.data_ptr(), _need(bias, "bias", (E,), _F32, dev), nt, T, E, k,
                         _code(logits.dtype, "logits"), score, n_groups, topk_groups, group_rule,
                         1 if renormalize else 0, scale)


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
    dev = _first(logits, "logits", 2)
    a = _topk_args(logits, dev, k, score, n_groups, topk_groups, group_rule, renormalize, scale, bias, n_tokens)
    T, E = logits.shape
    n = k if k > 0 else 0
    shapes = [("idx", (T, n), _I32), ("weights", (T, n), _F32), ("scores", (T, E), _F32 if want_scores else None)]
    if dispatch:
        slots = (T * n,)
        shapes += [("counts", (E,), _I32), ("offsets", (E + 1,), _I32), ("perm_token", slots, _I32),
                   ("perm_slot", slots, _I32), ("slot_pos", (T, n), _I32), ("gate_perm", slots, _F32)]
    given = out if out is not None else {}

    def call(handle):
        res, ptrs = {}, []
        for name, shape, dtype in shapes:
            if dtype is None:
                ptrs.append(None)
                continue
            t = given.get(name)
            if t is None:
                from torch import empty

                t = empty(shape, dtype=dtype, device=dev)
            res[name] = t
            ptrs.append(_need(t, name, shape, dtype, dev))
        if len(given) > len(res) or not given.keys() <= res.keys():
            _refuse(f"out holds {sorted(set(given) - set(res))}, which this call does not write")
        L = N.lib()
        ws, size = None, 0
        if workspace is not None:
            size = workspace.numel()
            ws = _need(workspace, "workspace", (size,), _U8, dev)
        elif dispatch and (size := L.moe_topk_workspace_size(T, E, n)):
            from torch import empty

            held = empty(size, dtype=_U8, device=dev)
            ws = held.data_ptr()
        _check(L.moe_topk_route(a, N.MoeTopkRouted(*ptrs), ws, size, handle), "moe_topk_route")
        return res

    return _on(dev, stream, call)


def moe_topk_route_backward(logits, idx, grad_weights, *, score=N.MOE_SCORE_SOFTMAX, renormalize=False, scale=1.0,
                            grad_scores=None, n_tokens=None, out=None, stream=None):
    """Gradient of moe_topk_route's ``weights`` (and ``scores``, if ``grad_scores`` [T, E]
    is given) to the logits, in the logits' type, for its choice ``idx``."""
    dev = _first(logits, "logits", 2)
    _first(idx, "idx", 2)
    k = idx.shape[1]
    a = _topk_args(logits, dev, k, score, 1, 1, N.MOE_GROUP_MAX, renormalize, scale, None, n_tokens)
    T, E = shape = logits.shape
    ip, gp = _need(idx, "idx", (T, k), _I32, dev), _need(grad_weights, "grad_weights", (T, k), _F32, dev)
    sp = _need(grad_scores, "grad_scores", shape, _F32, dev)

    def call(handle):
        g = out
        if g is None:
            from torch import empty_like

            g = empty_like(logits)
        _check(N.lib().moe_topk_route_backward(a, ip, gp, sp, _need(g, "out", shape, logits.dtype, dev), handle),
               "moe_topk_route_backward")
        return g

    return _on(dev, stream, call)


def moe_combine_topk(y, slot_pos, *, weights=None, residual=None, out=None, out_dtype=None, stream=None):
    """out[t] = residual[t] + sum_s weights[t, s] * y[slot_pos[t, s]] for rows y [R, d]
    and slot_pos [T, k] (int32; entries outside [0, R) add nothing). The output has
    ``out_dtype`` (bf16 or fp32), by default the residual's type, else y's."""
    dev = _first(y, "y", 2)
    _first(slot_pos, "slot_pos", 2)
    (R, d), (T, k) = y.shape, slot_pos.shape
    yc, pp = _code(y.dtype, "y"), _need(slot_pos, "slot_pos", (T, k), _I32, dev)
    wp = _need(weights, "weights", (T, k), _F32, dev)

    def call(handle):
        o = out
        if o is None:
            from torch import empty

            o = empty((T, d), dtype=out_dtype or (y.dtype if residual is None else residual.dtype), device=dev)
        elif out_dtype is not None and o.dtype is not out_dtype:
            _refuse(f"out has type {o.dtype}, not {out_dtype}")
        dtype = o.dtype
        oc = _code(dtype, "out")
        op, rp = _need(o, "out", (T, d), dtype, dev), _need(residual, "residual", (T, d), dtype, dev)
        _check(N.lib().moe_combine_topk(y.data_ptr(), yc, R, pp, wp, T, k, d, rp, op, oc, handle), "moe_combine_topk")
        return o

    return _on(dev, stream, call)
