"""The dense product with bias, activation and residual against a plain 64-bit form, within derived bounds."""
import math

import pytest
import torch

import block_quantized_routed_gb300 as moe

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
HALF_STEP = {F32: 2.0 ** -24, BF16: 2.0 ** -8, F16: 2.0 ** -11}
TINY = {F32: 2.0 ** -149, BF16: 2.0 ** -133, F16: 2.0 ** -25}
ACTS = {"none": moe.ACT_NONE, "relu": moe.ACT_RELU, "silu": moe.ACT_SILU, "gelu": moe.ACT_GELU, "gelu_tanh": moe.ACT_GELU_TANH}


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe.load()


def act64(y, act):
    if act == "relu":
        return y.clamp_min(0)
    if act == "silu":
        return y / (1 + torch.exp(-y))
    if act == "gelu":
        return 0.5 * y * torch.erfc(-y / math.sqrt(2))
    if act == "gelu_tanh":
        return 0.5 * y * (1 + torch.tanh(math.sqrt(2 / math.pi) * (y + 0.044715 * y ** 3)))
    return y


def reference(x, w, bias, act, residual, out_dtype):
    """The result and its bound: K additions of exact products, each off by a step (2^-23) of a partial sum at most
    (the tensor pipe may cut instead of round); activations with slopes below 1.13 and errors of 16 steps of their
    argument; the residual's addition; one rounding."""
    x, w = x.double(), w.double()
    y, A = x @ w.T, x.abs() @ w.abs().T
    if bias is not None:
        y, A = y + bias.double(), A + bias.double().abs()
    err = (x.shape[1] + 2) * 2.0 ** -23 * A
    if act != "none":
        err = 1.13 * err + 16 * 2.0 ** -23 * y.abs()
        y = act64(y, act)
    if residual is not None:
        y = y + residual.double()
        err = err + y.abs() * 2.0 ** -24
    return y, 1.01 * (err + y.abs() * HALF_STEP[out_dtype]) + TINY[out_dtype]


def run(T, N, K, dtype=BF16, act="none", bias=False, res=None, out=None, seed=0, strided=False, ws=None):
    g = torch.Generator(device="cuda").manual_seed(seed)
    out = out or dtype
    rnd = lambda *s, t=F32: torch.randn(*s, generator=g, device="cuda").to(t)
    pad = 8 if strided else 0
    x, w = rnd(T, K + pad, t=dtype)[:, :K], (rnd(N, K + 2 * pad) * K ** -0.5).to(dtype)[:, pad:K + pad]
    b = rnd(N) if bias else None
    r = (2 * rnd(T, N + 3 * strided)).to(res)[:, :N] if res else None
    o = torch.full((T + 1, N + 5 * strided), 7.0, dtype=out, device="cuda")
    moe.moe_linear(x, w, o[:T, :N], bias=b, act=ACTS[act], residual=r, ws=ws)
    y, tol = reference(x, w, b, act, r, out)
    assert (o[T:] == 7).all() and (o[:, N:] == 7).all()
    bad = (o[:T, :N].double() - y).abs() > tol
    if out == F16:
        bad &= ~((y.abs() + tol >= 65520) & torch.isinf(o[:T, :N]))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}, worst {((o[:T, :N].double() - y).abs() / tol).max():.2f} bounds"
    return x, w, o


@pytest.mark.parametrize("T", [1, 2, 7, 16, 17, 33, 64, 65, 100, 129])
@pytest.mark.parametrize("N,K", [(1, 8), (7, 64), (129, 72), (1000, 512), (5120, 2048), (2047, 4104), (384, 128)])
def test_few_tokens(T, N, K):
    run(T, N, K, BF16, seed=T)
    run(T, N, K, F16, act="silu", bias=True, res=F32, out=F32, seed=T + 1)


@pytest.mark.parametrize("T,N,K", [(200, 640, 1024), (257, 130, 200), (500, 4096, 256), (1021, 2049, 512), (3000, 256, 64),
                                   (2048, 2048, 2048), (777, 5000, 136), (4099, 100, 8)])
def test_many_tokens(T, N, K):
    run(T, N, K, BF16, bias=True, res=BF16, seed=T)
    run(T, N, K, F16, act="gelu", out=F32, seed=T + 1)


@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("dtype,res,out", [(BF16, None, BF16), (BF16, F32, F32), (BF16, BF16, F32), (F16, F16, F16), (F16, F32, F16)])
@pytest.mark.parametrize("T", [3, 150, 600])
def test_epilogues(act, dtype, res, out, T):
    run(T, 300, 192, dtype, act=act, bias=True, res=res, out=out, strided=True, seed=T)


def test_every_token_count_of_a_split():
    """Slices of the tokens are of unequal length, or empty."""
    for T in range(1, 36):
        run(T, 260, 1536, BF16, bias=True, seed=T)


def test_activations_far_out():
    """exp that overflows, tanh and erf that saturate."""
    x = torch.linspace(-200, 200, 1024, device="cuda").to(BF16).view(-1, 1) * torch.tensor([[1.0] + [0.0] * 7], device="cuda").to(BF16)
    w = torch.zeros(1, 8, dtype=BF16, device="cuda")
    w[0, 0] = 1
    for act, code in ACTS.items():
        out = torch.empty(1024, 1, device="cuda")
        moe.moe_linear(x.contiguous(), w, out, act=code)
        y = act64(x[:, :1].double(), act)
        # gelu's tails are differences of numbers near 1: off by steps of the argument
        assert ((out.double() - y).abs() <= 16 * 2.0 ** -23 * x[:, :1].double().abs() + 1e-37).all(), act


def test_residual_may_be_the_output():
    g = torch.Generator(device="cuda").manual_seed(1)
    for T in (5, 300):
        x, w = (torch.randn(n, 256, generator=g, device="cuda").to(BF16) for n in (T, 512))
        r = torch.randn(T, 512, generator=g, device="cuda")
        want = torch.empty_like(r)
        moe.moe_linear(x, w, want, residual=r)
        moe.moe_linear(x, w, r, residual=r)
        assert torch.equal(r, want)


@pytest.mark.parametrize("T", [4, 40, 300])
def test_numbers_that_are_not_finite_stay_in_their_row_and_column(T):
    g = torch.Generator(device="cuda").manual_seed(2)
    x, w = (torch.randn(n, 200, generator=g, device="cuda").to(BF16) for n in (T, 150))
    want = torch.empty(T, 150, device="cuda")
    moe.moe_linear(x, w, want)
    x[1, 3], w[7, 5], w[149, 199] = float("nan"), float("inf"), float("nan")
    got = torch.empty_like(want)
    moe.moe_linear(x, w, got)
    hit = torch.zeros(T, 150, dtype=torch.bool, device="cuda")
    hit[1] = hit[:, 7] = hit[:, 149] = True
    assert torch.equal(got[~hit], want[~hit]) and not torch.isfinite(got[hit]).any()


def test_results_repeat_on_streams_and_in_graphs():
    g = torch.Generator(device="cuda").manual_seed(3)
    for T, N, K in ((1, 5120, 2048), (37, 1000, 4096), (900, 1100, 512)):
        x, w = (torch.randn(n, K, generator=g, device="cuda").to(BF16) for n in (T, N))
        ws = torch.zeros(4, dtype=torch.int32, device="cuda")
        want, outs = torch.empty(T, N, device="cuda"), [torch.empty(T, N, device="cuda") for _ in range(3)]
        moe.moe_linear(x, w, want, ws=ws)
        torch.cuda.synchronize()
        for out in outs[:2]:
            s = torch.cuda.Stream()
            moe.moe_linear(x, w, out, stream=s)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            moe.moe_linear(x, w, outs[2], ws=ws)
        graph.replay()
        assert all(torch.equal(o, want) for o in outs) and not ws.any()
        x.neg_()
        graph.replay()
        assert torch.equal(outs[2], -want)


def test_no_tokens():
    out = torch.full((0, 64), 7.0, device="cuda")
    moe.moe_linear(torch.empty(0, 64, dtype=BF16, device="cuda"), torch.zeros(64, 64, dtype=BF16, device="cuda"), out)


def test_offsets_beyond_32_bits():
    """Rows of out, residual and x that start beyond 2^32 bytes."""
    T, N, K = 66000, 33000, 8
    g = torch.Generator(device="cuda").manual_seed(4)
    x, w = (torch.randn(n, K, generator=g, device="cuda").to(BF16) for n in (T, N))
    out = torch.zeros(T, N, dtype=BF16, device="cuda")
    out[-1] = 1.0
    moe.moe_linear(x, w, out, residual=out)
    for t in (0, T // 2, T - 300, T - 1):
        y, tol = reference(x[t:t + 1], w, None, "none", torch.full((1, N), float(t == T - 1), device="cuda"), BF16)
        assert ((out[t:t + 1].double() - y).abs() <= tol).all()
    wide = torch.zeros(3, 1 << 31, dtype=BF16, device="cuda")
    wide[:, :K] = x[:3]
    small = torch.empty(3, 64, device="cuda")
    moe.moe_linear(wide[:, :K], w[:64], small)
    y, tol = reference(x[:3], w[:64], None, "none", None, F32)
    assert ((small.double() - y).abs() <= tol).all()


def test_the_first_call_of_a_process_may_be_captured():
    """What the host asks of the device once does not disturb a capture."""
    code = """
import torch
import block_quantized_routed_gb300 as moe
x, w = torch.ones(3, 512, device="cuda").bfloat16(), torch.ones(700, 512, device="cuda").bfloat16()
big = torch.ones(900, 512, device="cuda").bfloat16()
out, out2 = torch.zeros(3, 700, device="cuda"), torch.zeros(900, 700, device="cuda")
torch.cuda.synchronize()
g = torch.cuda.CUDAGraph()
with torch.cuda.graph(g):
    moe.moe_linear(x, w, out)
    moe.moe_linear(big, w, out2)
g.replay()
torch.cuda.synchronize()
assert (out == 512).all() and (out2 == 512).all()
"""
    import subprocess
    import sys
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
