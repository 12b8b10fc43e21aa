"""The dense product on the CPU: refusals before any launch (no compute call is made here)."""
import ctypes

import pytest
import torch

import block_quantized_routed_gb300 as moe
from block_quantized_routed_gb300 import _build

FAKE = ctypes.c_void_p(0x10000)          # never dereferenced: validation fails first
ODD, OFF8 = ctypes.c_void_p(0x10001), ctypes.c_void_p(0x10008)
INV, UNS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.load()


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, x=None, w=None, out=None), 0), (dict(T=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(K=60, xs=64, wst=64), UNS),
    (dict(xt=0), UNS), (dict(xt=3), UNS), (dict(r=FAKE, rt=2), UNS), (dict(r=FAKE, rt=4), UNS), (dict(ot=2), UNS), (dict(ot=5), UNS),
    (dict(act=-1), UNS), (dict(act=5), UNS), (dict(x=None), INV), (dict(w=None), INV), (dict(out=None), INV), (dict(x=OFF8), INV),
    (dict(w=OFF8), INV), (dict(xs=56), INV), (dict(xs=68), INV), (dict(wst=56), INV), (dict(wst=68), INV), (dict(os=31), INV),
    (dict(r=FAKE, rt=1, rs=31), INV), (dict(b=ODD), INV), (dict(out=ODD), INV), (dict(r=ODD, rt=1, rs=32), INV), (dict(st=ODD), INV),
    (dict(wst=1 << 40), INV), (dict(T=1 << 30, N=1 << 20, os=1 << 20), UNS), (dict(T=2 ** 31 - 8, N=1, os=8), UNS),
    (dict(K=2 ** 31 - 8, xs=2 ** 31, wst=2 ** 31), UNS)])
def test_refusals(lib, kw, want):
    a = dict(x=FAKE, xt=1, xs=64, w=FAKE, wst=64, b=None, act=0, r=None, rt=0, rs=0, out=FAKE, ot=1, os=32, T=2, N=32, K=64, st=None)
    a.update(kw)
    assert lib.moe_linear(*a.values(), None) == want


def right():
    return dict(x=torch.zeros(3, 64, dtype=torch.bfloat16), w=torch.zeros(32, 64, dtype=torch.bfloat16),
                out=torch.zeros(3, 32), bias=torch.zeros(32), residual=torch.zeros(3, 32, dtype=torch.bfloat16),
                ws=torch.zeros(4, dtype=torch.uint8))


def test_tensors_of_the_host_are_refused(lib):
    with pytest.raises(moe.MoeError, match="GPU") as e:
        moe.moe_linear(**right())
    assert e.value.status == INV


@pytest.mark.parametrize("name,make", [
    ("x", lambda t: t[0]), ("x", lambda t: t[:, ::2]), ("w", lambda t: t.half()), ("w", lambda t: t[:, :32]), ("w", lambda t: t.t()),
    ("out", lambda t: t[:2]), ("out", lambda t: t[:, :16]), ("bias", lambda t: t[:8]), ("bias", lambda t: t.bfloat16()),
    ("residual", lambda t: t[:, :31]), ("ws", lambda t: t[:2]), ("x", lambda t: t.long()), ("w", lambda t: None)])
def test_wrong_tensors_are_refused(lib, name, make):
    a = right()
    with pytest.raises(moe.MoeError) as e:
        moe.moe_linear(**{**a, name: make(a[name])})
    assert "GPU" not in str(e.value)
