"""The 8-bit paged cache: codes and scales over all 16-bit numbers, layouts, roundings, and calls without rows."""
import numpy as np
import pytest
import torch

import block_quantized_routed_gb300 as moe
from tests.q8_ref import E4M3, INT8, Q8Cache, new_ws, quantise, status

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe.load()


@pytest.mark.parametrize("fmt", [E4M3, INT8])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_every_finite_number_is_a_largest_element(fmt, dtype):
    """A vector for each finite magnitude, the other elements any bits up to it: scales and codes are those of IEEE
    division, bit for bit."""
    top = 0x7f80 if dtype == torch.bfloat16 else 0x7c00
    g = torch.Generator().manual_seed(8)
    peak = torch.arange(top).unsqueeze(1)
    mag = torch.minimum((torch.rand(top, 63, generator=g, dtype=torch.float64) * (peak + 1)).long(), peak)
    mag[:, 32:] = (peak - torch.randint(0, 1500, (top, 31), generator=g)).clamp_min(0)    # near it: codes other than 0
    bits = torch.cat([peak, mag], 1) | torch.randint(0, 2, (top, 64), generator=g) << 15
    x = torch.from_numpy(bits.numpy().astype(np.uint16).view(np.int16)).view(dtype).view(top, 1, 64)
    c = Q8Cache([top], 1, 64, 64, fmt)
    ws, cu = new_ws(), torch.tensor([0, top], dtype=torch.int32).cuda()
    moe.moe_kv_append_q8(x.cuda(), x.flip(0).cuda(), c.gkc, c.gvc, c.gks, c.gvs, c.gtable, cu, c.kv_len, ws)
    assert status(ws) == 0
    ids = c.table[0].long()
    for v, codes, scales in ((x, c.gkc, c.gks), (x.flip(0), c.gvc, c.gvs)):
        want, d = quantise(v, fmt)
        got = codes.view(torch.uint8).cpu()[ids].view(-1, 1, 64)[:top]
        zero = (v == 0).all(-1)                                    # (zeros have code 0 whatever their sign)
        assert torch.equal(scales.cpu()[ids].view(-1, 1)[:top], d)
        assert torch.equal(got[~zero], want.view(torch.uint8)[~zero]) and not got[zero].any()


def test_keys_without_rows_are_told():
    """No rows at all: every key lies outside them."""
    c = Q8Cache([20, 0], 2, 64, 16, E4M3)
    first = torch.tensor([0, 20], dtype=torch.int32).cuda()
    out = torch.empty(0, 2, 64, device="cuda")
    for lens, want in (([20, 0], moe.MOE_ERR_DEVICE_BOUNDS), ([0, 3], moe.MOE_ERR_DEVICE_BOUNDS), ([0, -1], moe.MOE_ERR_DEVICE_BOUNDS),
                       ([0, 0], 0)):
        c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        ws = new_ws()
        moe.moe_kv_read_q8(c.gkc, c.gvc, c.gks, c.gvs, c.gtable, c.kv_len, first, out, out.clone(), ws)
        assert status(ws) == want, lens


def test_layouts_that_are_apart_are_taken():
    """Keys and values interleaved in one array, rows of every second place, scales of one array: none share memory.  A
    scale for the whole cache serves what reads it, and is refused where codes are written."""
    g = torch.Generator().manual_seed(4)
    both = torch.zeros(6, 2, 16, 4, 64, dtype=torch.uint8, device="cuda").view(E4M3)
    sc = torch.zeros(6, 4, 32, 2, device="cuda")
    kc, vc = both[:, 0, :, ::2], both[:, 1, :, 1::2]
    ks, vs = (sc[:, ::2, ::2, i].transpose(1, 2) for i in (0, 1))
    table, cu = torch.tensor([[4, 1, 3]], dtype=torch.int32).cuda(), torch.tensor([0, 40], dtype=torch.int32).cuda()
    kv_len, x = torch.tensor([40], dtype=torch.int32).cuda(), torch.randn(2, 40, 2, 64, generator=g).to(torch.bfloat16).cuda()
    ws = new_ws()
    moe.moe_kv_append_q8(x[0], x[1], kc, vc, ks, vs, table, cu, kv_len, ws)
    rows = torch.zeros(2, 40, 2, 64, device="cuda")
    moe.moe_kv_read_q8(kc, vc, ks, vs, table, kv_len, cu[:1], rows[0], rows[1], ws)
    assert status(ws) == 0
    d = x.float().abs().amax(-1, keepdim=True) / 448.0
    assert ((rows - x.float()).abs() <= torch.maximum(x.float().abs() * 2.0 ** -4, d * 2.0 ** -10) * (1 + 2.0 ** -10)).all()
    one = torch.full((1, 1, 1), 0.5, device="cuda").expand(6, 16, 2)
    with pytest.raises(moe.MoeError):
        moe.moe_kv_append_q8(x[0], x[1], kc, vc, one, vs, table, cu, kv_len, ws)
    moe.moe_kv_read_q8(kc, vc, one, one, table, kv_len, cu[:1], rows[0], rows[1], ws)
    ids = table[0].long()
    want = kc.view(torch.uint8)[ids].contiguous().view(E4M3).float().view(-1, 2, 64)[:40] * 0.5
    assert torch.equal(rows[0], want) and status(ws) == 0


@pytest.mark.parametrize("D", [64, 72])
def test_products_are_rounded_to_fp32_and_then_to_16_bits(D):
    """Scales whose product with the code 2.25 rounds to an fp32 number halfway between two of the output's: the second
    rounding goes by that number, half a step and 2^-24 off at most."""
    cases = {torch.bfloat16: [("0x1.a471c80000000p-1", 1.84375), ("0x1.29c71c0000000p-1", 1.3125), ("0x1.daaaaa0000000p-2", 1.046875)],
             torch.float16: [("0x1.1571c80000000p-1", 1.21875), ("0x1.64c71c0000000p-1", 1.568359375), ("0x1.be8e380000000p-1", 1.962890625)]}
    for dtype, pairs in cases.items():
        codes = torch.full((1, 16, 1, D), 0x41, dtype=torch.uint8, device="cuda").view(E4M3)
        scales = torch.ones(1, 16, 1, device="cuda")
        scales[0, :3, 0] = torch.tensor([float.fromhex(d) for d, _ in pairs])
        table, kv_len, first = (torch.tensor(t, dtype=torch.int32).cuda() for t in ([[0]], [3], [0]))
        out, ws = torch.zeros(2, 3, 1, D, dtype=dtype, device="cuda"), new_ws()
        moe.moe_kv_read_q8(codes, codes, scales, scales, table, kv_len, first, out[0], out[1], ws)
        assert status(ws) == 0
        for j, (d, want) in enumerate(pairs):
            assert (out[:, j].double() == want).all()
            exact = 2.25 * float.fromhex(d)
            assert abs(want - exact) <= torch.finfo(dtype).eps / 2 + 2.0 ** -24 * exact     # (values between 1 and 2)
