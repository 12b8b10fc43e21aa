"""MoeDecoderBlock: the operators run together.  Each stage is checked from the stage before it as the device left it:
attention and norms against 64-bit forms, the routed half against moe_layer_forward on the same normalised rows."""
import numpy as np
import pytest
import torch

import block_quantized_routed_gb300 as moe
import synth
from synth.layout import FMT_Q4K
from tests import block_ref
from tests.gpu_util import assert_close_rows, to_dev

pytestmark = pytest.mark.gpu
H, I, E, K, S = 512, 256, 16, 4, 1
HQ, HKV, D, PAGE = 8, 2, 64, 16


def make(route, T_max=64, seed=80, **kw):
    experts = [tuple(to_dev(synth.gen_matrix(FMT_Q4K, n, kk, seed, 0, e, m), torch) for m, (n, kk) in
                     enumerate([(I, H), (I, H), (H, I)])) for e in range(E + S)]
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s, scale=1.0: (torch.randn(s, generator=g) * scale)
    desc = dict(H=H, I=I, E=E, top_k=K, n_shared=S, route=route, fmt=FMT_Q4K, T_max=T_max)
    wr = to_dev(synth.router_weight(E, H, seed), torch)
    return moe.MoeDecoderBlock(desc, moe.expert_table(experts), (1 + 0.1 * rnd(H)).cuda(),
                               rnd((HQ + 2 * HKV) * D, H, scale=H ** -0.5).bfloat16().cuda(),
                               rnd(H, HQ * D, scale=(HQ * D) ** -0.5).bfloat16().cuda(), (1 + 0.1 * rnd(H)).cuda(), wr,
                               HQ, HKV, D, **kw), rnd


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe.load()


def lay(q_lens, kv_lens):
    need = [-(-k // PAGE) for k in kv_lens]
    table = torch.zeros(len(need), max(need), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = torch.arange(at, at + n, dtype=torch.int32)
        at += n
    cu = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32)
    return at + 1, table, cu, torch.tensor(kv_lens, dtype=torch.int32)


@pytest.mark.parametrize("route", [moe.ROUTE_SOFTMAX, moe.ROUTE_SIGMOID])
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [1]), ([1, 4, 20], [40, 4, 150]), ([33], [33])])
def test_block_stage_by_stage(route, q_lens, kv_lens):
    blk, rnd = make(route)
    pages, table, cu, kv = lay(q_lens, kv_lens)
    kc, vc = rnd(pages, PAGE, HKV, D).bfloat16().cuda(), rnd(pages, PAGE, HKV, D).bfloat16().cuda()
    T = int(cu[-1])
    x = rnd(T, H, scale=2.0).cuda()
    out = blk.forward(x, kc, vc, table.cuda(), cu.cuda(), kv.cuda())
    assert blk.status() == 0
    # attention over the cache as the call left it, with the new keys in place
    q = blk.qkv[:T].view(T, HQ + 2 * HKV, D).cpu()
    want, _, tol, _ = block_ref.attention(q[:, :HQ], kc.cpu(), vc.cpu(), table, q_lens, kv_lens, D ** -0.5, 0,
                                          torch.bfloat16)
    assert ((blk.attn[:T].view(T, HQ, D).cpu().double() - want).abs() <= tol).all()
    at = 0
    for b, (n, kvn) in enumerate(zip(q_lens, kv_lens)):
        for i in range(n):
            j = kvn - n + i
            p = int(table[b, j // PAGE])
            assert torch.equal(kc[p, j % PAGE].cpu(), q[at + i, HQ:HQ + HKV])
            assert torch.equal(vc[p, j % PAGE].cpu(), q[at + i, HQ + HKV:])
        at += n
    # the residual stream and its norm
    assert torch.equal(blk.resid[:T], blk.o[:T].float() + x)
    _, z = block_ref.norm(blk.o[:T].cpu(), x.cpu(), blk.ffn_norm.cpu(), blk.eps)
    assert ((blk.z[:T].cpu().double() - z).abs() <= 64 * 2.0 ** -24 * (z.abs() + 1e-3)).all()
    # the routed half: the layer entry point on the same rows chooses and computes the same
    layer = moe.MoeLayer(dict(H=H, I=I, E=E, top_k=K, n_shared=S, route=route, fmt=FMT_Q4K, T_max=64), blk.table,
                         blk.w_router)
    ids = torch.empty(T, K, dtype=torch.int32, device="cuda")
    ref = layer.forward(blk.z[:T].contiguous(), residual=blk.resid[:T].contiguous(), ids_out=ids)
    l = np.sort(blk.logits[:T].cpu().numpy(), axis=1)[:, ::-1]
    clear = np.abs(np.diff(l[:, :K + 1], axis=1)).min(axis=1) > 1e-4      # no near-tie between the two routers' sums
    assert clear.any()
    np.testing.assert_array_equal(ids.cpu().numpy()[clear], blk.ids[:T].cpu().numpy()[clear])
    assert_close_rows(out.cpu().numpy()[clear], ref.cpu().numpy()[clear], "block output")


def test_block_in_a_graph_and_in_place():
    """A decode step captured once and replayed as the sequences grow: kv_len advances on the device."""
    blk, rnd = make(moe.ROUTE_SIGMOID, router_bias=torch.linspace(-0.1, 0.1, E).cuda(), n_group=4, topk_group=2, scale=2.5)
    pages, table, cu, kv = lay([1, 1], [40, 25])
    mk = lambda: (torch.zeros(pages, PAGE, HKV, D, dtype=torch.bfloat16, device="cuda"),
                  torch.zeros(pages, PAGE, HKV, D, dtype=torch.bfloat16, device="cuda"))
    x0 = rnd(2, H).cuda()
    table, cu = table.cuda(), cu.cuda()

    def run(step_fn, caches, lens):
        res = []
        for _ in range(3):
            step_fn()
            res.append(step_fn.out.clone())
            lens.add_(1)
        return res

    kc, vc = mk()
    lens = torch.tensor([20, 5], dtype=torch.int32, device="cuda")
    eager = lambda: setattr(eager, "out", blk.forward(x0, kc, vc, table, cu, lens))
    want = run(eager, (kc, vc), lens)
    kc2, vc2 = mk()
    lens2 = torch.tensor([20, 5], dtype=torch.int32, device="cuda")
    x = x0.clone()
    out = torch.empty_like(x)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        blk.forward(x, kc2, vc2, table, cu, lens2, out=out)
    kc2.zero_(), vc2.zero_()
    replay = lambda: (graph.replay(), setattr(replay, "out", out))
    got = run(replay, (kc2, vc2), lens2)
    assert all(torch.equal(a, b) for a, b in zip(want, got))
    assert blk.status() == 0


def test_block_refuses_too_many_tokens():
    blk, rnd = make(moe.ROUTE_SOFTMAX, T_max=2)
    with pytest.raises(moe.MoeError):
        blk.forward(torch.zeros(3, H, device="cuda"), None, None, None, None, None)
