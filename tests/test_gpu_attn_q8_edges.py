"""Attention over an 8-bit paged cache where the work is laid out unusually or the scales are at the end of their range."""
import pytest
import torch

import block_quantized_routed_gb300 as moe
from tests.q8_ref import E4M3, INT8, Q8Cache, new_ws, status
from tests.test_gpu_attn_q8 import check, rnd

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe.load()


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("D", [64, 128, 256, 80])
def test_values_whose_scales_are_all_tiny(fmt, D):
    """Scales from 2^-126, the least that appending writes, to 2^-115: the results are normal numbers of bf16.  In one
    CTA, in parts that several join, and with a few keys of no value that hold most of the weight."""
    for lens, q_lens, heads in (([70, 9], [3, 1], 4), ([5000], [1], 8)):
        c = Q8Cache(lens, 1, D, 16, fmt, seed=D)
        g = torch.Generator().manual_seed(5)
        c.vs.copy_(torch.pow(2.0, -126 + 11 * torch.rand(c.vs.shape, generator=g)))
        c.gvs.copy_(c.vs)
        check(c, q_lens, heads)
        p0 = int(c.table[0, 0])
        c.vs[p0, :4] = 0.0
        c.ks[p0, :4] *= 8.0
        c.gvs.copy_(c.vs)
        c.gks.copy_(c.ks)
        check(c, q_lens, heads, seed=1)


@pytest.mark.parametrize("n,D,Hkv,G", [(600, 64, 1, 4), (300, 128, 2, 2), (150, 256, 1, 4), (150, 128, 1, 12)])
def test_more_sequences_than_threads_of_a_cta(n, D, Hkv, G):
    """Every thread looks after several sequences then; some have no new tokens, some no keys."""
    g = torch.Generator().manual_seed(n)
    lens = torch.randint(0, 200, (n,), generator=g).tolist()
    lens[n // 2] = 3000
    c = Q8Cache(lens, Hkv, D, 16, E4M3)
    check(c, [min(1, k) if i % 7 else 0 for i, k in enumerate(lens)], Hkv * G)
    check(c, [0] * (n - 1) + [min(lens[-1], 2)], Hkv * G, F16, seed=1)
    check(c, [min(k, 1 + i % 5) if i % 3 else 0 for i, k in enumerate(lens)], Hkv * G, window=50, seed=2)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("chunk", [100, 400])
def test_a_chunk_among_single_tokens(D, chunk):
    """One sequence of many new tokens beside many of one: the rows of an item go by the mean."""
    lens = [30 + 11 * i for i in range(40)] + [chunk + 300] + [5] * 8
    q_lens = [1] * 40 + [chunk] + [1] * 8
    c = Q8Cache(lens, 2, D, 16, INT8, seed=D)
    check(c, q_lens, 8)
    check(c, q_lens, 4, F16, window=130, seed=1)


def test_calls_that_overlap_repeat_calls_that_do_not():
    """Layers of a step, each call reading what the one before wrote, over buffers that later calls write again: the same
    bits as with the device waited for between the calls."""
    T, H, Hq, Hkv, D = 9, 512, 8, 2, 64
    g = torch.Generator().manual_seed(1)
    rand = lambda *s, scale=1.0: (scale * torch.randn(*s, generator=g)).to(BF16).cuda()
    w_qkv, w_o, w_up, w_down = (rand((Hq + 2 * Hkv) * D, H, scale=H ** -0.5), rand(H, Hq * D, scale=(Hq * D) ** -0.5),
                                rand(4 * H, H, scale=H ** -0.5), rand(H, 4 * H, scale=(4 * H) ** -0.5))
    x0 = rand(T, H)
    cu = torch.tensor([0, 1, 5, T], dtype=torch.int32).cuda()
    results = []
    for wait in (True, False):
        c = Q8Cache([3000, 70, 400], Hkv, D, 16, E4M3)
        x, qkv, o = x0.clone(), torch.empty(T, Hq + 2 * Hkv, D, dtype=BF16, device="cuda"), torch.empty(T, Hq, D, dtype=BF16, device="cuda")
        up, rows = torch.empty(T, 4 * H, dtype=BF16, device="cuda"), torch.empty(2, 4000, Hkv, D, dtype=BF16, device="cuda")
        first = torch.tensor([0, 3000, 3100], dtype=torch.int32).cuda()
        rows.zero_()
        ws = new_ws(moe.moe_paged_attention_q8_workspace_size(Hq, Hkv, D))
        torch.cuda.synchronize()
        sync = torch.cuda.synchronize if wait else lambda: None
        for _ in range(30):
            moe.moe_linear(x, w_qkv, qkv.view(T, -1), ws=ws)
            sync()
            moe.moe_kv_append_q8(qkv[:, Hq:Hq + Hkv], qkv[:, Hq + Hkv:], c.gkc, c.gvc, c.gks, c.gvs, c.gtable, cu, c.kv_len, ws)
            sync()
            moe.moe_paged_attention_q8(qkv[:, :Hq], c.gkc, c.gvc, c.gks, c.gvs, c.gtable, cu, c.kv_len, D ** -0.5, o, ws)
            sync()
            moe.moe_linear(o.view(T, -1), w_o, x, residual=x, ws=ws)
            sync()
            moe.moe_linear(x, w_up, up, act=moe.ACT_SILU, ws=ws)
            sync()
            moe.moe_linear(up, w_down, x, ws=ws)                       # (the residual stream starts again)
            sync()
            moe.moe_kv_read_q8(c.gkc, c.gvc, c.gks, c.gvs, c.gtable, c.kv_len, first, rows[0], rows[1], ws)
            sync()
        assert status(ws) == 0
        results.append([t.clone() for t in (x, qkv, o, up, rows, c.gkc.view(torch.uint8), c.gks)])
    assert all(torch.equal(a, b) for a, b in zip(*results)) and torch.isfinite(results[0][0].float()).all()


def test_operators_beside_one_another_on_streams():
    """Products of every kind, attention over both caches and the cache's own calls at one time, each stream with its own
    workspaces: the results of one after the other."""
    g = torch.Generator(device="cuda").manual_seed(3)
    rand = lambda *s: torch.randn(*s, generator=g, device="cuda").to(BF16)
    Hq, Hkv, D, n = 16, 2, 128, 4
    c = Q8Cache([5000, 800, 17, 2000], Hkv, D, 64, E4M3)
    k16, v16 = (rand(c.pages, 64, Hkv, D) for _ in range(2))
    q, cu = rand(n, Hq, D), torch.arange(n + 1, dtype=torch.int32).cuda()
    first = torch.tensor([0, 5000, 5800, 5817], dtype=torch.int32).cuda()
    xs = {t: (rand(t, 2048), rand(1100, 2048)) for t in (1, 40, 300, 1500)}

    def work():
        """The calls of a stream, their outputs and status words."""
        ws8, ws16, wl = (new_ws(b) for b in (moe.moe_paged_attention_q8_workspace_size(Hq, Hkv, D),
                                             moe.moe_paged_attention_workspace_size(Hq, Hkv, D), 16))
        o8, o16, rows = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(2, 7817, Hkv, D, dtype=BF16, device="cuda")
        ys = {t: torch.zeros(t, 1100, dtype=BF16, device="cuda") for t in xs}
        calls = [lambda t=t: moe.moe_linear(*xs[t], ys[t], ws=wl) for t in xs]
        calls.insert(1, lambda: moe.moe_paged_attention_q8(q, c.gkc, c.gvc, c.gks, c.gvs, c.gtable, cu, c.kv_len, 0.1, o8, ws8))
        calls.insert(3, lambda: moe.moe_paged_attention(q, k16, v16, c.gtable, cu, c.kv_len, 0.1, o16, ws16))
        calls.insert(5, lambda: moe.moe_kv_read_q8(c.gkc, c.gvc, c.gks, c.gvs, c.gtable, c.kv_len, first, rows[0], rows[1], wl))
        return calls, [o8, o16, rows, *ys.values()], (ws8, ws16, wl)
    calls, want, _ = work()
    for f in calls:
        f()
        torch.cuda.synchronize()
    streams, parts = [torch.cuda.Stream() for _ in range(3)], [work() for _ in range(3)]
    torch.cuda.synchronize()
    for i in range(60):
        for j, (s, (calls, _, _)) in enumerate(zip(streams, parts)):
            with torch.cuda.stream(s):
                calls[(i + 2 * j) % len(calls)]()
    torch.cuda.synchronize()
    for _, outs, spaces in parts:
        assert all(torch.equal(a, b) for a, b in zip(outs, want)) and [status(ws) for ws in spaces] == [0, 0, 0]
