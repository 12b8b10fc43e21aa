"""The 8-bit cache's operators on the CPU: refusals before any launch (no compute call is made here), and the plain
forms that the GPU tests compare with, pinned by hand-worked cases."""
import ctypes
import math

import numpy as np
import pytest
import torch

import block_quantized_routed_gb300 as moe
from block_quantized_routed_gb300 import _build
from tests.q8_ref import E4M3, INT8, code_values, quantise

FAKE = ctypes.c_void_p(0x10000)          # never dereferenced: validation fails first
ODD = ctypes.c_void_p(0x10001)
OFF8 = ctypes.c_void_p(0x10004)
INV, UNS, WS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return moe.load()


def desc(**kw):
    d = dict(n_seqs=2, Hkv=2, D=64, dtype=moe.DT_E4M3, page_size=16, num_pages=8, max_pages=4, reserved=0, table_stride=4,
             k_page_stride=2048, k_row_stride=128, k_head_stride=64, v_page_stride=2048, v_row_stride=128, v_head_stride=64)
    d.update(kw)
    return ctypes.byref(moe.KvDesc(**d))


def scales(**kw):
    d = dict(k=0x20000, v=0x30000, k_page_stride=32, k_row_stride=1, k_head_stride=16, v_page_stride=32, v_row_stride=1,
             v_head_stride=16)
    d.update(kw)
    return ctypes.byref(moe.KvScales(**d))


def append_rc(lib, **kw):
    a = dict(kv=desc(), sc=scales(), xt=1, k=FAKE, ks=128, kh=64, v=FAKE, vs=128, vh=64, kc=FAKE, vc=FAKE, table=FAKE,
             cu=FAKE, len=FAKE, T=2, ws=FAKE, n=16)
    a.update(kw)
    return lib.moe_kv_append_q8(*a.values(), None)


KV_REFUSALS = [(dict(kv=None), INV), (dict(kv=desc(dtype=1)), UNS), (dict(kv=desc(dtype=5)), UNS),
               (dict(kv=desc(D=60)), UNS), (dict(kv=desc(D=264)), UNS), (dict(kv=desc(n_seqs=0)), UNS),
               (dict(kv=desc(page_size=0)), INV), (dict(kv=desc(reserved=1)), INV), (dict(kv=desc(k_row_stride=-1)), INV),
               (dict(kv=desc(table_stride=3)), INV), (dict(kv=desc(max_pages=1 << 28, table_stride=1 << 28)), UNS),
               (dict(sc=None), INV), (dict(sc=scales(k=None)), INV), (dict(sc=scales(v=0x20002)), INV),
               (dict(sc=scales(v_head_stride=-1)), INV), (dict(ws=None), INV), (dict(n=15), WS), (dict(ws=ODD), INV),
               (dict(table=None), INV), (dict(len=ODD), INV)]


@pytest.mark.parametrize("kw,want", KV_REFUSALS + [
    (dict(T=0, k=None, ws=None, sc=None), 0), (dict(T=-1), INV), (dict(xt=0), UNS), (dict(xt=3), UNS), (dict(k=None), INV),
    (dict(k=ODD), INV), (dict(v=ODD), INV), (dict(ks=-8), INV), (dict(vh=-8), INV), (dict(cu=None), INV),
    (dict(kc=None), INV)])
def test_append_refusals(lib, kw, want):
    assert append_rc(lib, **kw) == want


def read_rc(lib, **kw):
    a = dict(kv=desc(), sc=scales(), kc=FAKE, vc=FAKE, table=FAKE, len=FAKE, first=FAKE, rows=8, ot=1, ko=FAKE, ks=128,
             kh=64, vo=FAKE, vs=128, vh=64, ws=FAKE, n=16)
    a.update(kw)
    return lib.moe_kv_read_q8(*a.values(), None)


@pytest.mark.parametrize("kw,want", KV_REFUSALS + [
    (dict(rows=0, ko=None, ws=None, sc=None), 0), (dict(rows=-1), INV), (dict(ot=3), UNS), (dict(ot=-1), UNS),
    (dict(ko=None), INV), (dict(ko=ODD), INV), (dict(ot=0, vo=ctypes.c_void_p(0x10002)), INV), (dict(first=None), INV),
    (dict(first=ODD), INV), (dict(ks=64), INV), (dict(kh=63), INV), (dict(vs=0), INV), (dict(vh=0), INV)])
def test_read_refusals(lib, kw, want):
    assert read_rc(lib, **kw) == want


def attn_rc(lib, **kw):
    n = lib.moe_paged_attention_q8_workspace_size(4, 2, 64)
    a = dict(kv=desc(), sc=scales(), xt=1, q=FAKE, qs=256, qh=64, Hq=4, T=2, kc=FAKE, vc=FAKE, table=FAKE, cu=FAKE,
             len=FAKE, scale=0.1, window=0, out=FAKE, os=256, oh=64, lse=None, ws=FAKE, n=n)
    a.update(kw)
    return lib.moe_paged_attention_q8(*a.values(), None)


@pytest.mark.parametrize("kw,want", KV_REFUSALS + [
    (dict(T=0, q=None, ws=None, sc=None), 0), (dict(T=-1), INV), (dict(xt=0), UNS), (dict(Hq=5), UNS), (dict(Hq=0), INV),
    (dict(Hq=2048), UNS), (dict(T=1 << 30), UNS), (dict(window=-1), INV), (dict(scale=math.inf), INV),
    (dict(scale=math.nan), INV), (dict(q=None), INV), (dict(q=OFF8), INV), (dict(out=OFF8), INV), (dict(qs=100), INV),
    (dict(oh=4), INV), (dict(kc=OFF8), INV), (dict(kv=desc(v_row_stride=132)), INV), (dict(lse=ODD), INV),
    (dict(n=0), WS)])
def test_attention_refusals(lib, kw, want):
    assert attn_rc(lib, **kw) == want


def test_attention_workspace_sizes(lib):
    size = moe.moe_paged_attention_q8_workspace_size
    assert size(8, 2, 128) >= 16 and size(4, 2, 80) >= 16
    assert size(5, 2, 128) == size(8, 2, 60) == size(8, 0, 128) == size(2048, 2, 128) == size(8, 2, 264) == 0


def calls():
    """Each operator with tensors that are right but for their device."""
    for fmt in (E4M3, INT8):
        kc = torch.zeros(8, 16, 2, 64, dtype=torch.uint8).view(fmt)
        ks = torch.zeros(8, 16, 2)
        table, cu = torch.zeros(2, 4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
        n, kn = torch.zeros(2, dtype=torch.int32), torch.zeros(3, 2, 64, dtype=torch.bfloat16)
        ws = torch.zeros(1 << 12, dtype=torch.uint8)
        q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
        a = dict(k=kn, v=kn, k_cache=kc, v_cache=kc, k_scale=ks, v_scale=ks, page_table=table, cu_q=cu, kv_len=n, ws=ws)
        yield moe.moe_kv_append_q8, a
        yield moe.moe_kv_read_q8, dict(k_cache=kc, v_cache=kc, k_scale=ks, v_scale=ks, page_table=table, kv_len=n, first=n,
                                       k_out=kn, v_out=kn, ws=ws)
        yield moe.moe_paged_attention_q8, dict(q=q, k_cache=kc, v_cache=kc, k_scale=ks, v_scale=ks, page_table=table,
                                               cu_q=cu, kv_len=n, scale=0.1, out=q.clone(), ws=ws, lse=torch.zeros(3, 4))


def test_tensors_of_the_host_are_refused(lib):
    for f, a in calls():
        with pytest.raises(moe.MoeError, match="GPU") as e:
            f(**a)
        assert e.value.status == INV


@pytest.mark.parametrize("name,make", [
    ("k_cache", lambda t: t.to(torch.bfloat16)), ("v_cache", lambda t: t[:4]), ("k_scale", lambda t: t.double()),
    ("v_scale", lambda t: t.transpose(1, 2)), ("k_scale", lambda t: t[:4]), ("page_table", lambda t: t.long()),
    ("kv_len", lambda t: t[:1]), ("cu_q", lambda t: t[:2]), ("first", lambda t: t.float()), ("ws", lambda t: t[::2]),
    ("k", lambda t: t[..., :32]), ("k", lambda t: t.float()[:, :1]), ("v", lambda t: t.half()), ("v", lambda t: t[:2]),
    ("v_out", lambda t: t.float()), ("k_out", lambda t: t[..., ::2]), ("q", lambda t: t[..., :56]),
    ("out", lambda t: t.half()), ("out", lambda t: t[:, :2]), ("lse", lambda t: t.t()), ("lse", lambda t: t.double()),
    ("k_cache", lambda t: 3)])
def test_wrong_tensors_are_refused(lib, name, make):
    hit = 0
    for f, a in calls():
        if name in a:
            hit += 1
            with pytest.raises(moe.MoeError) as e:
                f(**{**a, name: make(a[name])})
            assert "GPU" not in str(e.value)
    assert hit


def test_plain_quantiser_by_hand():
    x = torch.tensor([[448.0, 17.0, 19.0, -21.0, 2.0 ** -10, 3 * 2.0 ** -10, 0.0, -448.0]])
    codes, d = quantise(x, E4M3)
    assert d.item() == 1.0 and codes.float().tolist() == [[448.0, 16.0, 20.0, -20.0, 0.0, 2.0 ** -8, 0.0, -448.0]]
    codes, d = quantise(torch.tensor([[254.0, 1.0, 3.0, -1.0, -3.0, 0.5, -254.0, 0.0]]), INT8)
    assert d.item() == 2.0 and codes.tolist() == [[127, 1, 2, -1, -2, 0, -127, 0]]
    for fmt in (E4M3, INT8):
        codes, d = quantise(torch.tensor([[0.0, -0.0], [math.nan, 1.0], [1.0, -math.inf]]), fmt)
        assert d[0] == 0 and torch.isnan(d[1:]).all() and not codes.view(torch.uint8).any()
        assert quantise(torch.tensor([[2.0 ** -133]]), fmt)[1].item() == 2.0 ** -126


def test_values_of_the_e4m3_codes():
    codes = torch.arange(256).to(torch.uint8).view(E4M3)
    assert np.array_equal(code_values(codes).numpy(), codes.float().double().numpy(), equal_nan=True)
