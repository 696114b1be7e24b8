"""Refusals of moe_int8_product: on the host, before any launch. No GPU."""

import ctypes

import pytest
import torch

import mixture_experts_ffn_14_b200 as moe
from mixture_experts_ffn_14_b200 import _native as N
from mixture_experts_ffn_14_b200 import build as B

BASE = 0x10000000  # never dereferenced


@pytest.fixture(scope="module", autouse=True)
def built_library():
    B.build()
    return N.lib()


def args(**kw):
    a = N.MoeInt8Args(BASE, None, None, BASE, BASE, None, BASE, None, None, BASE, 64, 64, 256, 512, 8, N.MOE_BF16,
                      N.MOE_BF16, 0)
    for name, v in kw.items():
        setattr(a, name, v)
    return a


def call(ws=BASE * 2, ws_bytes=1 << 40, **kw):
    return N.lib().moe_int8_product(ctypes.byref(args(**kw)), ws, ws_bytes, None)


@pytest.mark.parametrize("change", [
    dict(R=-1), dict(K=0), dict(N=0), dict(n_experts=0), dict(x_dtype=N.MOE_BF16_INT8W), dict(x_dtype=9),
    dict(out_dtype=N.MOE_INT8), dict(x_rows=-1), dict(x_rows=63), dict(x=None), dict(w=None), dict(s=None),
    dict(out=None), dict(w_up=BASE), dict(s_up=BASE), dict(counts=None), dict(x_scale=BASE),
    dict(x_dtype=N.MOE_INT8), dict(x_dtype=N.MOE_INT8, x_scale=BASE, index=BASE),
    dict(w_up=BASE, s_up=BASE, activation=3)])
def test_invalid(change):
    assert call(**change) == N.MOE_ERR_INVALID_ARG


@pytest.mark.parametrize("change", [dict(K=264), dict(N=520), dict(K=131072), dict(N=(1 << 20) + 16),
                                    dict(R=(1 << 24) + 1, x_rows=(1 << 24) + 1), dict(n_experts=1025)])
def test_unsupported(change):
    assert call(**change) == N.MOE_ERR_UNSUPPORTED
    size = {"R": 64, "K": 256, "N": 512, "n_experts": 8}
    size.update({k: v for k, v in change.items() if k in size})
    assert moe.moe_int8_workspace_size(size["R"], size["K"], size["N"], size["n_experts"]) == 0


def test_alignment_and_workspace():
    for name in ("x", "counts", "w", "s", "out", "gate", "index"):
        assert call(**{name: BASE + 8}) == N.MOE_ERR_MISALIGNED, name
    assert call(ws=None) == N.MOE_ERR_WORKSPACE
    assert call(ws=BASE + 16) == N.MOE_ERR_WORKSPACE
    assert call(ws_bytes=moe.moe_int8_workspace_size(64, 256, 512, 8) - 1) == N.MOE_ERR_WORKSPACE
    assert N.lib().moe_int8_product(None, None, 0, None) == N.MOE_ERR_INVALID_ARG
    assert call(R=0, x_rows=0, x=None, out=None, ws=None) == N.MOE_OK
    assert moe.moe_int8_workspace_size(0, 256, 512, 8) == 0
    assert moe.moe_int8_workspace_size(64, 256, 512, 8, N.MOE_INT8) < moe.moe_int8_workspace_size(64, 256, 512, 8)
    assert N.lib().moe_int8_workspace_size(64, 256, 512, 8, N.MOE_BF16, 2) == 0


def test_binding_refuses():
    x, w, s = torch.zeros(4, 32), torch.zeros(1, 32, 16, dtype=torch.int8), torch.zeros(1, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        moe.moe_int8_product(x, w, s)                   # host tensors
    with pytest.raises(ValueError):
        moe.moe_int8_product(x.half(), w, s)
    with pytest.raises(ValueError):
        moe.moe_int8_product(x, w[0], s)
    with pytest.raises(ValueError):
        moe.moe_int8_product(x, w, s, w_up=w)
