"""Refusals of the routing and combine calls of any E and k: on the host, before
any launch, through the C ABI and through the binding. No GPU."""

import ctypes

import pytest
import torch

import mixture_experts_ffn_14_b200 as moe
from mixture_experts_ffn_14_b200 import _native as N
from mixture_experts_ffn_14_b200 import build as B

BASE = 0x10000000  # never dereferenced: every call returns from its checks


@pytest.fixture(scope="module", autouse=True)
def built_library():
    B.build()
    return N.lib()


def args(T=400, E=16, k=2, dtype=N.MOE_F32, score=0, n_groups=1, topk_groups=1, rule=0, renorm=0, scale=1.0,
         logits=BASE, bias=None, n_tokens=None):
    return N.MoeTopkArgs(logits, bias, n_tokens, T, E, k, dtype, score, n_groups, topk_groups, rule, renorm, scale)


def routed(**kw):
    r = N.MoeTopkRouted(*[BASE + 0x1000 * i for i in range(1, 10)])
    for name, v in kw.items():
        setattr(r, name, v)
    return r


def call(a, r=None, ws=BASE * 2, ws_bytes=1 << 30):
    r = routed() if r is None else r
    return N.lib().moe_topk_route(ctypes.byref(a), ctypes.byref(r), ws, ws_bytes, None)


@pytest.mark.parametrize("change,status", [
    (dict(T=-1), N.MOE_ERR_INVALID_ARG), (dict(E=0), N.MOE_ERR_INVALID_ARG), (dict(k=0), N.MOE_ERR_INVALID_ARG),
    (dict(k=17), N.MOE_ERR_INVALID_ARG), (dict(dtype=N.MOE_BF16_INT8W), N.MOE_ERR_INVALID_ARG),
    (dict(score=2), N.MOE_ERR_INVALID_ARG), (dict(renorm=2), N.MOE_ERR_INVALID_ARG),
    (dict(scale=float("nan")), N.MOE_ERR_INVALID_ARG), (dict(scale=float("inf")), N.MOE_ERR_INVALID_ARG),
    (dict(n_groups=0), N.MOE_ERR_INVALID_ARG), (dict(n_groups=3), N.MOE_ERR_INVALID_ARG),
    (dict(n_groups=4, topk_groups=5), N.MOE_ERR_INVALID_ARG), (dict(n_groups=4, topk_groups=0), N.MOE_ERR_INVALID_ARG),
    (dict(rule=2), N.MOE_ERR_INVALID_ARG), (dict(E=1025), N.MOE_ERR_UNSUPPORTED),
    (dict(E=128, k=33), N.MOE_ERR_UNSUPPORTED), (dict(E=128, n_groups=64), N.MOE_ERR_UNSUPPORTED),
    (dict(T=(1 << 24) + 1), N.MOE_ERR_UNSUPPORTED), (dict(logits=None), N.MOE_ERR_INVALID_ARG),
    (dict(logits=BASE + 4), N.MOE_ERR_MISALIGNED), (dict(bias=BASE + 8), N.MOE_ERR_MISALIGNED),
    (dict(n_tokens=BASE + 2), N.MOE_ERR_MISALIGNED),
])
def test_route_refuses(change, status):
    assert call(args(**change)) == status


def test_route_refuses_outputs_and_workspace():
    assert call(args(), routed(idx=None)) == N.MOE_ERR_INVALID_ARG
    assert call(args(), routed(weights=None)) == N.MOE_ERR_INVALID_ARG
    assert call(args(), routed(counts=None)) == N.MOE_ERR_INVALID_ARG        # some of the dispatch arrays
    assert call(args(), routed(slot_pos=BASE + 8)) == N.MOE_ERR_MISALIGNED
    assert call(args(), routed(scores=BASE + 8)) == N.MOE_ERR_MISALIGNED
    assert call(args(), ws=None) == N.MOE_ERR_WORKSPACE
    assert call(args(), ws=BASE + 16) == N.MOE_ERR_WORKSPACE
    assert call(args(), ws_bytes=100) == N.MOE_ERR_WORKSPACE
    assert N.lib().moe_topk_route(None, None, None, 0, None) == N.MOE_ERR_INVALID_ARG
    assert N.lib().moe_topk_route(ctypes.byref(args()), None, None, 0, None) == N.MOE_ERR_INVALID_ARG
    bare = N.MoeTopkRouted()
    assert call(args(T=0, logits=None), bare, ws=None, ws_bytes=0) == N.MOE_OK


def test_workspace_size():
    size = moe.moe_topk_workspace_size
    assert size(0, 8, 2) == size(-1, 8, 2) == size(64, 2000, 2) == size(64, 8, 9) == 0
    assert size(256, 256, 8) == 0                     # one launch: nothing kept between kernels
    assert size(257, 256, 8) >= 9 * 256 * 4 and size(257, 256, 8) % 256 == 0
    assert size(1 << 24, 1024, 8) > (1 << 24) // 32 * 1024 * 4   # past 32 bits


def test_backward_refuses():
    def f(a, idx=BASE, gw=BASE, gs=None, out=BASE):
        return N.lib().moe_topk_route_backward(ctypes.byref(a), idx, gw, gs, out, None)

    assert f(args(T=0)) == N.MOE_OK
    assert f(args(k=33, E=64)) == N.MOE_ERR_UNSUPPORTED
    assert f(args(score=5)) == N.MOE_ERR_INVALID_ARG
    assert f(args(), idx=None) == f(args(), gw=None) == f(args(), out=None) == N.MOE_ERR_INVALID_ARG
    assert f(args(), gs=BASE + 4) == f(args(), out=BASE + 2) == N.MOE_ERR_MISALIGNED


def test_combine_refuses():
    def f(y=BASE, yd=N.MOE_F32, R=10, pos=BASE, w=None, T=4, k=2, d=64, res=None, out=BASE, od=N.MOE_BF16):
        return N.lib().moe_combine_topk(y, yd, R, pos, w, T, k, d, res, out, od, None)

    assert f(T=0) == N.MOE_OK
    for bad in (dict(T=-1), dict(R=-1), dict(k=0), dict(d=0), dict(yd=2), dict(od=2), dict(y=None), dict(pos=None),
                dict(out=None)):
        assert f(**bad) == N.MOE_ERR_INVALID_ARG, bad
    for bad in (dict(d=60), dict(k=33), dict(T=(1 << 24) + 1), dict(R=(1 << 29) + 1)):
        assert f(**bad) == N.MOE_ERR_UNSUPPORTED, bad
    for bad in (dict(y=BASE + 8), dict(out=BASE + 8), dict(res=BASE + 8), dict(w=BASE + 4), dict(pos=BASE + 4)):
        assert f(**bad) == N.MOE_ERR_MISALIGNED, bad


def test_binding_refuses_host_tensors():
    l = torch.zeros(4, 8)
    with pytest.raises(ValueError):
        moe.moe_topk_route(l, 2)
    with pytest.raises(ValueError):
        moe.moe_topk_route(torch.zeros(8), 2)
    with pytest.raises(ValueError):
        moe.moe_topk_route_backward(l, torch.zeros(4, 2, dtype=torch.int32), torch.zeros(4, 2))
    with pytest.raises(ValueError):
        moe.moe_combine_topk(l, torch.zeros(4, 2, dtype=torch.int32))
