"""The dense product on every plan, whatever sizes the choice by cost would take it for: rings that wrap, last blocks of
terms, tokens and features that are not whole, several tiles to a CTA."""
import pytest
import torch

import block_quantized_routed_gb300 as moe
from tests.test_gpu_linear import ACTS, reference

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
SINGLE = [(16, 1), (32, 1), (64, 1), (128, 1), (256, 1), (128, 0), (256, 0)]
SHARED = [(t, c) for t in (16, 32, 64, 128) for c in range(2, 9)]
KINDS = [(act, res, out) for act in ACTS for res, out in ((None, "x"), ("x", "x"), (F32, F32), (None, F32), (F32, "x"))]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe.load()


def check(T, N, K, plan, n, dtype):
    act, res, out = KINDS[n % len(KINDS)]
    res, out = dtype if res == "x" else res, dtype if out == "x" else out
    g = torch.Generator(device="cuda").manual_seed(n)
    rnd = lambda *s, t=F32: torch.randn(*s, generator=g, device="cuda").to(t)
    x, w = rnd(T, K, t=dtype), (rnd(N, K) * K ** -0.5).to(dtype)
    b = rnd(N) if n % 3 else None
    r = (2 * rnd(T, N)).to(res) if res else None
    o, ws = torch.full((T + 1, N + 3), 7.0, dtype=out, device="cuda"), torch.zeros(4, dtype=torch.int32, device="cuda")
    moe.moe_debug_linear(x, w, o[:T, :N], *plan, bias=b, act=ACTS[act], residual=r, ws=ws)
    y, tol = reference(x, w, b, act, r, out)
    assert (o[T:] == 7).all() and (o[:, N:] == 7).all() and not ws.any()
    err = (o[:T, :N].double() - y).abs()
    assert (err <= tol).all(), f"{int((err > tol).sum())} of {err.numel()}, worst {(err / tol).max():.2f} bounds"
    # the plan changes the order of the sums alone
    moe.moe_linear(x, w, o[:T, :N], bias=b, act=ACTS[act], residual=r, ws=ws)
    assert ((o[:T, :N].double() - y).abs() <= tol).all()


@pytest.mark.parametrize("plan", SINGLE + SHARED, ids=str)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_edges(plan, dtype):
    """More blocks of terms to a CTA than any ring holds, the last of 8; features and tokens that end in either half."""
    t, c = plan
    K = 64 * 13 * max(1, c) + 8
    n = 7 * (SINGLE + SHARED).index(plan) + (dtype == F16)
    for i, (T, N) in enumerate([(1, 1), (t - 1, 300), (t + 5, 456), (t + t // 2 + 3, 127), (2 * t, 256), (2 * t + 9, 517)]):
        check(T, N, K, plan, n + i, dtype)


@pytest.mark.parametrize("plan", SINGLE, ids=str)
@pytest.mark.parametrize("K", [8, 64, 200, 1096])
def test_several_tiles_of_a_cta(plan, K):
    """The accumulators' turns and the ring go on from tile to tile."""
    t, c = plan
    tiles = 25 if t <= 32 else 12
    check(t * tiles - t // 2 - 5, 3999, K, plan, K + t + c, BF16 if t % 3 else F16)


def test_plans_that_are_none():
    x, w, out = torch.zeros(4, 128, dtype=BF16, device="cuda"), torch.zeros(8, 128, dtype=BF16, device="cuda"), torch.zeros(4, 8, device="cuda")
    for plan in ((0, 1), (48, 1), (512, 1), (16, 0), (64, 0), (256, 2), (16, 9), (16, 3), (128, -1)):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_debug_linear(x, w, out, *plan)
        assert e.value.status == moe.MOE_ERR_UNSUPPORTED
