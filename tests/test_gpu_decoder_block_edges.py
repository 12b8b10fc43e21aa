"""MoeDecoderBlock beyond its ordinary step: errors and what follows them, strided tensors, the caller's settings, the
rotary function and the window."""
import numpy as np
import pytest
import torch

import block_quantized_routed_gb300 as moe
from tests import block_ref
from tests.test_gpu_decoder_block import D, E, H, HKV, HQ, PAGE, lay, make

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe.load()


def step(blk, rnd, q_lens, kv_lens, x=None, out=None, seed=5):
    """One call over a cache of random keys: (out, x, cache, table, cu, kv)."""
    pages, table, cu, kv = lay(q_lens, kv_lens)
    g = torch.Generator().manual_seed(seed)
    kc, vc = (torch.randn(pages, PAGE, HKV, D, generator=g).bfloat16().cuda() for _ in range(2))
    if x is None:
        x = (2.0 * torch.randn(int(cu[-1]), H, generator=g)).cuda()
    return blk.forward(x, kc, vc, table.cuda(), cu.cuda(), kv.cuda(), out=out), x, (kc, vc), table, cu, kv


def test_status_reads_every_workspace():
    """An error in two workspaces is told once, not again by the next call."""
    blk, rnd = make(moe.ROUTE_SIGMOID)
    step(blk, rnd, [1, 3], [40, 20])
    assert blk.status() == 0
    for ws, code in ((blk.attn_ws, moe.MOE_ERR_DEVICE_BOUNDS), (blk.ffn_ws, moe.MOE_ERR_DEVICE_TIMEOUT)):
        ws[:4].view(torch.int32).fill_(code)
    assert blk.status() == moe.MOE_ERR_DEVICE_BOUNDS
    assert blk.status() == 0


def test_block_after_a_wait_that_ran_out():
    """Attention gives up waiting for the parts of a long sequence; the next step is right."""
    blk, rnd = make(moe.ROUTE_SIGMOID)
    want = step(blk, rnd, [1], [6000])[0].clone()
    assert blk.status() == 0
    counters = blk.attn_ws[16:16 + 4 * 160].view(torch.int32)
    counters.fill_(2 ** 30)                                  # an increment takes these to 0: the parts never add up
    step(blk, rnd, [1], [6000])
    assert blk.status() == moe.MOE_ERR_DEVICE_TIMEOUT
    assert (counters == 0).all()
    assert torch.equal(step(blk, rnd, [1], [6000])[0], want) and blk.status() == 0


def test_out_with_a_stride():
    """x and out as columns of wider tensors, and out in place: rows go where they belong and nowhere else."""
    blk, rnd = make(moe.ROUTE_SIGMOID)
    want, x = step(blk, rnd, [1, 6], [40, 30])[:2]
    want = want.clone()
    T = x.shape[0]
    wide = torch.full((T, H + 13), 7.0, device="cuda")
    out = wide[:, 5:5 + H]
    assert step(blk, rnd, [1, 6], [40, 30], x=x, out=out)[0] is out
    assert torch.equal(out, want) and (wide[:, :5] == 7).all() and (wide[:, 5 + H:] == 7).all()
    wide = torch.full((T, H + 8), 7.0, device="cuda")
    xs = wide[:, 4:4 + H]
    xs.copy_(x)
    step(blk, rnd, [1, 6], [40, 30], x=xs, out=xs)
    assert torch.equal(xs, want) and (wide[:, :4] == 7).all() and (wide[:, 4 + H:] == 7).all()
    flat = torch.full((T * H + 1,), 7.0, device="cuda")      # rows without gaps, off the 16-byte boundary
    step(blk, rnd, [1, 6], [40, 30], x=x, out=flat[1:].view(T, H))
    assert torch.equal(flat[1:].view(T, H), want) and flat[0] == 7
    assert blk.status() == 0


def test_out_of_another_shape_or_type_is_refused():
    blk, rnd = make(moe.ROUTE_SIGMOID)
    for out in (torch.empty(7, H + 1, device="cuda"), torch.empty(6, H, device="cuda"),
                torch.empty(7, H, device="cuda", dtype=torch.bfloat16), torch.empty(7, H)):
        with pytest.raises(moe.MoeError):
            step(blk, rnd, [1, 6], [40, 30], out=out)


SWITCHES = {"allow_tf32": lambda: setattr(torch.backends.cuda.matmul, "allow_tf32", True),
            "precision": lambda: torch.set_float32_matmul_precision("high"),
            "fp32_precision": lambda: setattr(torch.backends.cuda.matmul, "fp32_precision", "tf32"),
            "off": lambda: None}


@pytest.mark.parametrize("switch", list(SWITCHES))
@pytest.mark.parametrize("q_lens,kv_lens", [([1], [30]), ([1, 50], [40, 50]), ([150], [200])])
def test_routing_does_not_follow_the_callers_tf32_switch(q_lens, kv_lens, switch):
    """Router logits are fp32 products of the normalised rows: choices depend on them."""
    if switch == "fp32_precision" and not hasattr(torch.backends.cuda.matmul, "fp32_precision"):
        pytest.skip("no such switch")
    blk, rnd = make(moe.ROUTE_SIGMOID, T_max=256)
    T = sum(q_lens)
    try:
        SWITCHES[switch]()
        step(blk, rnd, q_lens, kv_lens)
    finally:
        if hasattr(torch.backends.cuda.matmul, "fp32_precision"):
            torch.backends.cuda.matmul.fp32_precision = "ieee"
        torch.set_float32_matmul_precision("highest")
    z, logits = blk.z[:T].contiguous(), blk.logits[:T]
    want = torch.empty_like(logits)
    if switch == "off":
        torch.matmul(z, blk.w_router.t(), out=want)
    else:
        moe.moe_route_topk(z, blk.w_router, None, 4, moe.ROUTE_SIGMOID, want,
                           torch.empty(T, 4, dtype=torch.int32, device="cuda"), torch.empty(T, 4, device="cuda"))
    assert torch.equal(logits, want)
    # H products and sums in fp32 in any order; the split of long chunks' operands keeps 2^-22 of each
    bound = (z.double().abs() @ blk.w_router.double().abs().t()) * (H * 2.0 ** -24 + 2.0 ** -20)
    assert ((logits.double() - z.double() @ blk.w_router.double().t()).abs() <= bound).all()
    assert blk.status() == 0


def test_router_weights_of_another_layout_or_type():
    blk, rnd = make(moe.ROUTE_SIGMOID)
    want = step(blk, rnd, [3], [20])[0].clone()
    args = (blk.desc, blk.table, blk.attn_norm, blk.w_qkv, blk.w_o, blk.ffn_norm)
    other = moe.MoeDecoderBlock(*args, blk.w_router.t().contiguous().t(), HQ, HKV, D)
    assert torch.equal(step(other, rnd, [3], [20])[0], want)
    for w in (blk.w_router.bfloat16(), blk.w_router[:-1]):
        with pytest.raises(moe.MoeError):
            moe.MoeDecoderBlock(*args, w, HQ, HKV, D)


@pytest.mark.parametrize("window", [0, 7, 40])
def test_rotary_and_window(window):
    """The caller's rotation of new queries and keys by their positions comes before the cache and the attention; the
    window limits what the attention sees."""
    def rotary(q, k, cu, kv):
        n, t = cu[1:] - cu[:-1], torch.arange(q.shape[0], device="cuda", dtype=torch.int32)
        seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
        pos = (kv - n)[seq] + t - cu[seq]
        freq = 0.3 ** torch.arange(D // 2, device="cuda")
        ang = pos[:, None, None] * freq
        for v in (q, k):
            a, b = v[..., :D // 2].float(), v[..., D // 2:].float()
            v.copy_(torch.cat([a * ang.cos() - b * ang.sin(), a * ang.sin() + b * ang.cos()], -1))
        rotary.seen = (q.clone(), k.clone())

    blk, rnd = make(moe.ROUTE_SIGMOID, rotary=rotary, window=window)
    q_lens, kv_lens = [1, 4, 20], [40, 4, 150]
    out, x, (kc, vc), table, cu, kv = step(blk, rnd, q_lens, kv_lens)
    assert blk.status() == 0
    T = int(cu[-1])
    q, k = (t.cpu() for t in rotary.seen)
    want, _, tol, _ = block_ref.attention(q, kc.cpu(), vc.cpu(), table, q_lens, kv_lens, D ** -0.5, window, torch.bfloat16)
    assert ((blk.attn[:T].view(T, HQ, D).cpu().double() - want).abs() <= tol).all()
    for b, (n, kvn) in enumerate(zip(q_lens, kv_lens)):
        for i in range(n):
            j, t = kvn - n + i, int(cu[b]) + i
            assert torch.equal(kc[int(table[b, j // PAGE]), j % PAGE].cpu(), k[t])
    plain = moe.MoeDecoderBlock(blk.desc, blk.table, blk.attn_norm, blk.w_qkv, blk.w_o, blk.ffn_norm, blk.w_router, HQ, HKV, D)
    assert not torch.equal(step(plain, rnd, q_lens, kv_lens)[0], out)
