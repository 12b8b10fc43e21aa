"""The decoder-block operators on the CPU: refusals before any launch (no compute call is made here), and the
plain 64-bit forms that the GPU tests compare with, pinned by hand-worked cases."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_quantized_routed_gb300 as moe
from block_quantized_routed_gb300 import _build
from tests import block_ref

FAKE = ctypes.c_void_p(0x10000)          # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10001)
INV, UNS, WS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.load()


def norm_rc(lib, **kw):
    a = dict(x=FAKE, xt=1, xs=512, r=None, rt=0, rs=0, w=FAKE, wt=0, off=0.0, eps=1e-6, T=2, H=512, s=None, ss=0,
             y=FAKE, yt=1, ys=512, fmt=0, q=None, d=None, bs=None)
    a.update(kw)
    return lib.moe_add_rmsnorm(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, x=None, w=None, y=None), 0), (dict(T=-1), INV), (dict(H=0), INV), (dict(H=16640), UNS),
    (dict(eps=-1.0), INV), (dict(eps=math.nan), INV), (dict(x=None), INV), (dict(w=None), INV), (dict(y=None), INV),
    (dict(xt=3), UNS), (dict(wt=-1), UNS), (dict(yt=7), UNS), (dict(r=FAKE, rt=2, rs=512), UNS),
    (dict(xs=511), INV), (dict(r=FAKE, rt=1, rs=100), INV), (dict(ys=0), INV), (dict(s=FAKE, ss=1), INV),
    (dict(fmt=5), UNS), (dict(fmt=1), INV), (dict(fmt=1, q=FAKE), INV), (dict(fmt=1, H=320, q=FAKE, d=FAKE), UNS),
    (dict(fmt=2, q=FAKE, d=FAKE, bs=FAKE), INV), (dict(x=ODD), INV), (dict(y=ODD), INV),
    (dict(fmt=1, q=FAKE, d=ODD), INV)])
def test_norm_refusals(lib, kw, want):
    assert norm_rc(lib, **kw) == want


def route_rc(lib, **kw):
    a = dict(l=FAKE, dt=0, st=64, b=None, T=2, E=64, k=4, route=1, ng=1, kg=1, gs=1, ren=1, sc=1.0, ids=FAKE, g=FAKE)
    a.update(kw)
    return lib.moe_route_grouped(*a.values(), None)


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, l=None, ids=None), 0), (dict(T=-1), INV), (dict(E=0), INV), (dict(k=0), INV), (dict(k=17), UNS),
    (dict(E=1025, st=1025), UNS), (dict(E=3, k=4), UNS), (dict(route=2), UNS), (dict(gs=2), UNS), (dict(dt=3), UNS),
    (dict(ng=0), INV), (dict(kg=0), INV), (dict(ng=5), UNS), (dict(ng=64), UNS), (dict(ng=4, kg=5), UNS),
    (dict(ng=32, kg=1), UNS), (dict(st=63), INV), (dict(l=None), INV), (dict(ids=None), INV), (dict(g=None), INV),
    (dict(l=ODD), INV), (dict(ids=ODD), INV), (dict(b=ODD), INV)])
def test_route_refusals(lib, kw, want):
    assert route_rc(lib, **kw) == want


def kv(**kw):
    a = dict(n_seqs=2, Hkv=2, D=64, dtype=1, page_size=16, num_pages=8, max_pages=4, reserved=0, table_stride=4,
             k_page_stride=2048, k_row_stride=128, k_head_stride=64, v_page_stride=2048, v_row_stride=128,
             v_head_stride=64)
    a.update(kw)
    return moe.KvDesc(**a)


def append_rc(lib, desc=None, **kw):
    a = dict(k=FAKE, ks=128, kh=64, v=FAKE, vs=128, vh=64, kc=FAKE, vc=FAKE, tab=FAKE, cu=FAKE, len=FAKE, T=3, ws=FAKE,
             n=16)
    a.update(kw)
    return lib.moe_kv_append(desc if desc is not None else kv(), *a.values(), None)


def attn_rc(lib, desc=None, **kw):
    a = dict(q=FAKE, qs=256, qh=64, Hq=4, T=3, kc=FAKE, vc=FAKE, tab=FAKE, cu=FAKE, len=FAKE, scale=0.1, win=0,
             out=FAKE, os=256, oh=64, lse=None, ws=FAKE, n=1 << 40)
    a.update(kw)
    return lib.moe_paged_attention(desc if desc is not None else kv(), *a.values(), None)


BAD_KV = [(dict(n_seqs=0), UNS), (dict(n_seqs=8193), UNS), (dict(Hkv=0), UNS), (dict(D=0), UNS), (dict(D=12), UNS),
          (dict(D=264), UNS), (dict(dtype=0), UNS), (dict(page_size=0), INV), (dict(num_pages=0), INV),
          (dict(max_pages=0), INV), (dict(reserved=1), INV), (dict(table_stride=3), INV), (dict(k_row_stride=-128), INV),
          (dict(page_size=1 << 20, max_pages=1 << 12, table_stride=1 << 12), UNS)]


@pytest.mark.parametrize("kw,want", BAD_KV)
def test_cache_desc_refusals(lib, kw, want):
    assert append_rc(lib, kv(**kw)) == want
    assert attn_rc(lib, kv(**kw)) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, k=None, ws=None), 0), (dict(T=-1), INV), (dict(k=None), INV), (dict(vc=None), INV), (dict(tab=None), INV),
    (dict(len=None), INV), (dict(ws=None), INV), (dict(n=8), WS), (dict(k=ODD), INV), (dict(ws=ODD), INV),
    (dict(ks=-1), INV)])
def test_append_refusals(lib, kw, want):
    assert append_rc(lib, **kw) == want


@pytest.mark.parametrize("kw,want", [
    (dict(T=0, q=None, ws=None), 0), (dict(T=-1), INV), (dict(Hq=3), UNS), (dict(Hq=0), INV), (dict(win=-1), INV),
    (dict(scale=math.inf), INV), (dict(scale=math.nan), INV), (dict(q=None), INV), (dict(out=None), INV),
    (dict(cu=None), INV), (dict(q=ODD), INV), (dict(out=ctypes.c_void_p(0x10008)), INV), (dict(qs=252), INV),
    (dict(oh=60), INV), (dict(lse=ODD), INV), (dict(ws=ctypes.c_void_p(0x10010)), INV), (dict(n=255), WS),
    (dict(Hq=1024, T=1 << 22), UNS)])
def test_attention_refusals(lib, kw, want):
    assert attn_rc(lib, **kw) == want


def test_attention_cache_strides_refused(lib):
    for name in ("k_page_stride", "k_row_stride", "k_head_stride", "v_page_stride", "v_row_stride", "v_head_stride"):
        assert attn_rc(lib, kv(**{name: 2052})) == INV      # rows off 16-byte boundaries


def test_attention_work_limit(lib):
    """A million tokens of 128 heads over a table of a million keys could be 2^31 tiles and more: refused."""
    d = kv(n_seqs=1, Hkv=8, D=128, page_size=64, max_pages=1 << 14, num_pages=1 << 14, table_stride=1 << 14)
    assert attn_rc(lib, d, Hq=128, qs=16384, os=16384, T=1 << 20) == UNS


def test_attention_workspace_size(lib):
    assert moe.moe_paged_attention_workspace_size(32, 8, 128) >= 256
    for bad in [(0, 1, 64), (3, 2, 64), (4, 2, 60), (4, 2, 512), (4, 0, 64)]:
        assert moe.moe_paged_attention_workspace_size(*bad) == 0


def test_binding_refuses_wrong_tensors():
    """Shape, stride and type checks of the Python binding come before any device work: CPU tensors reach them."""
    x = torch.zeros(2, 64)
    w = torch.ones(64)
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm(x, torch.ones(63), 1e-6, y=x.clone())
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm(x, w, 1e-6, y=torch.zeros(2, 65))
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm(x, w, 1e-6, y=torch.zeros(64, 2).t())
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm(x.double(), w, 1e-6, y=x.clone())
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm(x, w, 1e-6, residual=x, sum_out=x.half())
    with pytest.raises(moe.MoeError):
        moe.moe_add_rmsnorm(x, w, 1e-6, q_fmt=moe.NORM_Q_INT8_ROW, q=torch.zeros(2, 64, dtype=torch.int8))
    ids, gates = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(2, 4)
    with pytest.raises(moe.MoeError):
        moe.moe_route_grouped(x, 5, ids, gates)
    with pytest.raises(moe.MoeError):
        moe.moe_route_grouped(x, 4, ids, gates, bias=torch.zeros(63))
    kc = torch.zeros(8, 16, 2, 64, dtype=torch.bfloat16)
    tab, cu, n = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    ws = torch.zeros(64, dtype=torch.uint8)
    kn = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError):
        moe.moe_kv_append(kn.half(), kn, kc, kc, tab, cu, n, ws)
    with pytest.raises(moe.MoeError):
        moe.moe_kv_append(kn, kn, kc, kc, tab, cu[:2], n, ws)
    with pytest.raises(moe.MoeError):
        moe.moe_kv_append(kn, kn[:2], kc, kc, tab, cu, n, ws)
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(moe.MoeError):
        moe.moe_paged_attention(q, kc, kc, tab, cu, n, 0.1, q[:2], ws)
    with pytest.raises(moe.MoeError):
        moe.moe_paged_attention(q, kc, kc, tab, cu, n, 0.1, torch.empty_like(q), ws, lse=torch.zeros(3, 5))


# ------------------------------------------------------------------ the plain forms

def test_plain_norm_by_hand():
    s, z = block_ref.norm(torch.tensor([[3.0, 4.0]]), torch.tensor([[0.0, 0.0]]), torch.tensor([1.0, 2.0]), 0.0)
    r = math.sqrt(12.5)
    assert torch.allclose(z, torch.tensor([[3 / r, 8 / r]], dtype=torch.float64))
    _, z = block_ref.norm(torch.zeros(1, 4), None, torch.ones(4), 1e-6, offset=1.0)
    assert (z == 0).all()


def test_plain_route_by_hand():
    l = np.array([[0.0, 2.0, 1.0, 3.0]], np.float32)
    ids, g = block_ref.route(l, None, 2, False, 1, 1, True, True, 1.0)
    assert ids.tolist() == [[3, 1]]
    assert np.allclose(g, [[1 / (1 + math.exp(-1)), 1 / (1 + math.exp(1))]])
    # the bias chooses, the gates do not see it; equal keys go to the lower index
    ids, g = block_ref.route(l * 0, np.array([0, 1, 1, 0], np.float32), 2, True, 1, 1, True, False, 2.0)
    assert ids.tolist() == [[1, 2]] and np.allclose(g, 1.0)
    # groups {0,1} and {2,3}: best single expert in the second, best pair in the first
    l = np.array([[1.0, 1.0, -9.0, 1.5]], np.float32)
    assert block_ref.route(l, None, 1, True, 2, 1, True, True, 1.0)[0].tolist() == [[0]]
    assert block_ref.route(l, None, 1, True, 2, 1, False, True, 1.0)[0].tolist() == [[3]]
    ids, g = block_ref.route(np.full((1, 3), -np.inf, np.float32), None, 2, False, 1, 1, True, True, 1.0)
    assert ids.tolist() == [[0, 1]] and (g == 0).all()


def test_plain_attention_by_hand():
    # two keys of one page, scores 0 and ln 3: weights 1/4 and 3/4
    q = torch.tensor([[[1.0]], [[1.0]]])
    k = torch.tensor([0.0, math.log(3.0), 9.0, 9.0]).view(1, 4, 1, 1)
    v = torch.tensor([4.0, 8.0, math.nan, math.nan]).view(1, 4, 1, 1)
    out, lse, *_ = block_ref.attention(q, k, v, torch.zeros(1, 1, dtype=torch.int32), [2], [2], 1.0, 0, torch.float32)
    assert torch.allclose(out.flatten(), torch.tensor([4.0, 7.0], dtype=torch.float64))
    assert torch.allclose(lse.flatten(), torch.tensor([0.0, math.log(4.0)], dtype=torch.float64), atol=1e-7)
    # a window of one key sees the last key alone; a sequence without keys gives 0 and -inf
    out, lse, *_ = block_ref.attention(q, k, v, torch.zeros(1, 1, dtype=torch.int32), [2], [2], 1.0, 1, torch.float32)
    assert torch.allclose(out.flatten(), torch.tensor([4.0, 8.0], dtype=torch.float64))
    out, lse, *_ = block_ref.attention(q, k, v, torch.zeros(1, 1, dtype=torch.int32), [2], [0], 1.0, 0, torch.float32)
    assert (out == 0).all() and torch.isneginf(lse).all()
