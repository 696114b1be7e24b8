"""Routing, its gradient and the combine of any number of experts and choices
per token: Python binding of the C calls of the same names (include/moe.h).

Every tensor is dense, on one CUDA device, which need not be the current one;
the work goes to ``stream`` (a torch stream or a handle), by default that
device's current stream. Outputs and workspaces that are not given are allocated
on that stream. Wrong shapes, types and devices raise ``ValueError``, a call that
the library refuses ``MoeError``; no kernel of the library is launched in either case.

The calls are no part of an autograd graph: their results require no gradient, whatever
their inputs do (the weights' and scores' gradient is moe_topk_route_backward). A tensor
given as an output counts as changed in place for autograd.

    r = moe.moe_topk_route(logits, 8, score=moe.MOE_SCORE_SIGMOID, bias=bias, renormalize=True)
    ...                                  # experts on rows r["perm_token"], gates r["gate_perm"]
    out = moe.moe_combine_topk(y, r["slot_pos"])
"""

from __future__ import annotations

import ctypes

from . import _native as N

__all__ = ["moe_topk_route", "moe_topk_route_backward", "moe_topk_workspace_size", "moe_combine_topk"]

_calls = None  # module _torch_calls once loaded (the package imports without torch)


def _load():
    """The calls on tensors (csrc/torch_calls.cpp), set up for the loaded library."""
    global _calls
    import torch  # noqa: F401  (its libraries, which the module is linked against)

    try:
        from . import _torch_calls
    except ImportError as e:
        raise RuntimeError("mixture_experts_ffn_14_b200/_torch_calls.so cannot be loaded: build it with "
                           "`python -m mixture_experts_ffn_14_b200.build`") from e
    from . import MoeError

    L = N.lib()
    _torch_calls.setup(MoeError, *(ctypes.cast(f, ctypes.c_void_p).value for f in (
        L.moe_topk_workspace_size, L.moe_topk_route, L.moe_topk_route_backward, L.moe_combine_topk,
        L.moe_int8_workspace_size, L.moe_int8_product)))
    _calls = _torch_calls
    return _calls


def _on(stream, t, call, args):
    """Run call(*args) with `stream` (torch stream or handle) current, so that what the
    call allocates belongs to it, too."""
    import torch

    if not t.is_cuda:
        raise ValueError("moe: tensors must live on a CUDA device")
    s = stream
    if isinstance(stream, int):  # ExternalStream(0) would be a new stream, not the default one
        s = torch.cuda.ExternalStream(stream, device=t.device) if stream else torch.cuda.default_stream(t.device)
    if s.device != t.device:
        raise ValueError(f"moe: stream is on {s.device}, the tensors on {t.device}")
    with torch.cuda.stream(s):
        return call(*args)


def moe_topk_workspace_size(T, E, k) -> int:
    """Workspace bytes of moe_topk_route with the dispatch (0: none needed)."""
    return N.lib().moe_topk_workspace_size(T, E, k)


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
    call = (_calls or _load()).topk_route
    args = (logits, k, score, bias, n_groups, topk_groups, group_rule, renormalize, scale, n_tokens, want_scores,
            dispatch, out, workspace)
    return call(*args) if stream is None else _on(stream, logits, call, args)


def moe_topk_route_backward(logits, idx, grad_weights, *, score=N.MOE_SCORE_SOFTMAX, renormalize=False, scale=1.0,
                            grad_scores=None, n_tokens=None, out=None, stream=None):
    """Gradient of moe_topk_route's ``weights`` (and ``scores``, if ``grad_scores`` [T, E]
    is given) to the logits, in the logits' type, for its choice ``idx``."""
    call = (_calls or _load()).topk_route_backward
    args = (logits, idx, grad_weights, score, renormalize, scale, grad_scores, n_tokens, out)
    return call(*args) if stream is None else _on(stream, logits, call, args)


def moe_combine_topk(y, slot_pos, *, weights=None, residual=None, out=None, out_dtype=None, stream=None):
    """out[t] = residual[t] + sum_s weights[t, s] * y[slot_pos[t, s]] for rows y [R, d]
    and slot_pos [T, k] (int32; entries outside [0, R) add nothing). The output has
    ``out_dtype`` (bf16 or fp32), by default the residual's type, else y's."""
    call = (_calls or _load()).combine_topk
    args = (y, slot_pos, weights, residual, out, out_dtype)
    return call(*args) if stream is None else _on(stream, y, call, args)
