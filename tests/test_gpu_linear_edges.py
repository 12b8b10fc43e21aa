"""The dense product where its arrays lie among one another, and its activations over all numbers."""
import pytest
import torch

import block_quantized_routed_gb300 as moe
from tests.test_gpu_linear import reference

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe.load()


@pytest.mark.parametrize("T", [1, 5, 300])
def test_columns_of_one_buffer(T):
    """x, residual and out as columns of one array with one stride are apart, a single row of out in the gap of w's rows too."""
    K, N = 128, 96
    g = torch.Generator(device="cuda").manual_seed(T)
    buf = torch.randn(T, K + 2 * N, generator=g, device="cuda").to(BF16)
    w = torch.randn(N, K, generator=g, device="cuda").to(BF16)
    x, r, out = buf[:, :K], buf[:, K:K + N], buf[:, K + N:]
    y, tol = reference(x, w, None, "none", r, BF16)
    keep = buf[:, :K + N].clone()
    moe.moe_linear(x, w, out, residual=r)
    assert ((out.double() - y).abs() <= tol).all() and torch.equal(buf[:, :K + N], keep)
    for bad in (buf[:, K - 1:K - 1 + N], buf[:, 0:N]):
        with pytest.raises(moe.MoeError):
            moe.moe_linear(x, w, bad, residual=r)
    if T == 1:
        wide = torch.randn(N, K + N, generator=g, device="cuda").to(BF16)
        y, tol = reference(x, wide[:, :K], None, "none", None, BF16)
        moe.moe_linear(x, wide[:, :K], wide[3:4, K:])
        assert ((wide[3:4, K:].double() - y).abs() <= tol).all()


def test_residuals_that_are_not_quite_out_are_refused():
    x, w = torch.ones(8, 64, dtype=BF16, device="cuda"), torch.ones(32, 64, dtype=BF16, device="cuda")
    out = torch.zeros(9, 32, device="cuda")
    for r in (out.view(BF16)[:8, :32], out.view(BF16).view(-1)[:256].view(8, 32), out[1:9]):
        with pytest.raises(moe.MoeError) as e:
            moe.moe_linear(x, w, out[:8], residual=r)
        assert e.value.status == moe.MOE_ERR_INVALID_ARG
    assert not out.any()
    moe.moe_linear(x, w, out[:8], residual=out[:8])
    assert (out[:8] == 64).all() and not out[8].any()


def test_silu_of_every_number_that_it_holds():
    """2^-20 + |v| 2^-23 of itself: the exponential of a rounded argument within 2 ulp, a quotient within 2 ulp."""
    bits = torch.arange(1 << 16).int()
    v = bits.where(bits < 1 << 15, bits - (1 << 16)).short().view(BF16)
    v = v[torch.isfinite(v) & (v > -87)]
    x = torch.zeros(len(v), 8, dtype=BF16, device="cuda")
    x[:, 0] = v.cuda()
    w = torch.zeros(1, 8, dtype=BF16, device="cuda")
    w[0, 0] = 1
    out = torch.empty(len(v), 1, device="cuda")
    moe.moe_linear(x, w, out, act=moe.ACT_SILU)
    d = v.double()
    want = d / (1 + torch.exp(-d))
    err = (out[:, 0].cpu().double() - want).abs()
    assert (err <= (2.0 ** -20 + d.abs() * 2.0 ** -23) * want.abs() + 2.0 ** -126).all()
