"""The dense product's refusals of outputs that lie in its inputs and of plans that are none (before any launch; no compute
call is made here)."""
import ctypes

import pytest

import block_quantized_routed_gb300 as moe
from block_quantized_routed_gb300 import _build

INV = moe.MOE_ERR_INVALID_ARG
X, W, OUT = 0x100000, 0x200000, 0x300000          # never dereferenced: validation fails first


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.load()


# x [4, 64] and w [32, 64] of bf16 with rows of 128 bytes, out [4, 32]
@pytest.mark.parametrize("kw", [
    dict(out=X), dict(out=X + 3 * 128 + 126), dict(out=X - 3 * 64 - 62), dict(out=W + 31 * 128), dict(out=W - 2),
    dict(ot=0, out=X - 3 * 128 - 124, os=32), dict(x=X, xs=128, out=X + 64, os=128), dict(x=X, xs=128, out=X + 254, os=128),
    dict(x=X, xs=128, out=X + 256 + 66, os=128), dict(x=X, xs=128, out=X - 256 + 256 - 62, os=128), dict(x=X, xs=128, out=X + 128, os=100),
    dict(T=1, w=W, wst=128, out=W + 5 * 256 + 126), dict(T=1, w=W, wst=128, out=W + 5 * 256 - 62), dict(b=OUT + 100),
    dict(b=OUT - 124), dict(st=OUT + 4),
    # a residual in the place of out but for its type, its stride or a shift
    dict(r=OUT, rt=0, ot=1), dict(r=OUT, rt=1, ot=0), dict(r=OUT, rt=1, rs=40), dict(r=OUT + 2, rt=1), dict(r=OUT + 64, rt=1, rs=32),
    dict(r=OUT - 62, rt=1, rs=64, os=64), dict(T=1, r=OUT + 62, rt=1)])
def test_out_in_an_input_is_refused(lib, kw):
    a = dict(x=X, xt=1, xs=64, w=W, wst=64, b=None, act=0, r=None, rt=1, rs=32, out=OUT, ot=1, os=32, T=4, N=32, K=64, st=None)
    a.update(kw)
    for name in ("x", "w", "b", "r", "out", "st"):
        a[name] = ctypes.c_void_p(a[name]) if a[name] else None
    assert lib.moe_linear(*a.values(), None) == INV


@pytest.mark.parametrize("tokens,ctas,T,N,K", [(0, 1, 4, 32, 64), (48, 1, 4, 32, 64), (512, 1, 4, 32, 64), (16, 0, 4, 32, 64),
                                               (64, 0, 4, 32, 64), (256, 2, 4, 32, 512), (16, 9, 4, 32, 1024), (16, 3, 4, 32, 128),
                                               (128, -1, 4, 32, 64), (16, 1, 1 << 20, 1 << 20, 64)])
def test_plans_that_are_none_are_refused(lib, tokens, ctas, T, N, K):
    p = [ctypes.c_void_p(x) for x in (X, W, OUT)]
    assert lib.moe_debug_linear(p[0], 1, K, p[1], K, None, 0, None, 1, 0, p[2], 1, N, T, N, K, tokens, ctas, None,
                                None) == moe.MOE_ERR_UNSUPPORTED
