"""Writing and reading an 8-bit paged cache, against the definition in IEEE fp32: codes, scales and values bit for bit."""
import pytest
import torch

import block_quantized_routed_gb300 as moe
from tests.q8_ref import E4M3, INT8, Q8Cache, code_values, new_ws, quantise, status

pytestmark = pytest.mark.gpu
BF16, F16, F32 = torch.bfloat16, torch.float16, torch.float32
FMTS = [E4M3, INT8]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe.load()


def raw(t):
    return t.view(torch.uint8) if t.dtype == E4M3 else t


def check_append(c, q_lens, k, v, gk=None, gv=None):
    """Appends k, v [T, Hkv, D] as the last q_lens tokens of the sequences; everything else has to stay."""
    cu = torch.tensor([0] + q_lens).cumsum(0).int()
    ws = new_ws()
    moe.moe_kv_append_q8(k.cuda() if gk is None else gk, v.cuda() if gv is None else gv, c.gkc, c.gvc, c.gks, c.gvs,
                         c.gtable, cu.cuda(), c.kv_len, ws)
    assert status(ws) == 0
    want = {}
    for name, x, codes, scales in (("k", k, c.kc, c.ks), ("v", v, c.vc, c.vs)):
        q, d = quantise(x, c.fmt)
        codes, scales = raw(codes).clone(), scales.clone()
        for b, n in enumerate(q_lens):
            for i in range(n):
                pos = c.lens[b] - n + i
                page = int(c.table[b, pos // c.page])
                codes[page, pos % c.page] = raw(q)[cu[b] + i]
                scales[page, pos % c.page] = d[cu[b] + i]
        want[name] = codes, scales
    for (codes, scales), gc, gs in zip(want.values(), (c.gkc, c.gvc), (c.gks, c.gvs)):
        assert torch.equal(raw(gc).cpu(), codes)
        assert torch.equal(gs.cpu().view(torch.int32) & 0x7fffffff, scales.view(torch.int32) & 0x7fffffff) or \
            torch.equal(torch.nan_to_num(gs.cpu(), nan=-1.0), torch.nan_to_num(scales, nan=-1.0))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("Hkv,D,page", [(8, 128, 16), (1, 256, 64), (3, 64, 48), (2, 80, 1), (5, 8, 7), (1, 24, 16)])
def test_append(fmt, dtype, Hkv, D, page):
    lens, q = [37, 1, 64, 5], [5, 1, 0, 3]
    for layout in ("rows", "heads", "odd"):
        c = Q8Cache(lens, Hkv, D, page, fmt, seed=D, layout=layout)
        g = torch.Generator().manual_seed(1)
        x = torch.randn(sum(q), 3 * Hkv, D, generator=g).to(dtype)
        gx = x.cuda()
        check_append(c, q, x[:, :Hkv], x[:, Hkv:2 * Hkv], gx[:, :Hkv], gx[:, Hkv:2 * Hkv])  # views with strides


@pytest.mark.parametrize("fmt", FMTS)
def test_append_many_tokens(fmt):
    lens = [777, 300, 1, 1200] + [40] * 60
    q = [700, 300, 1, 1] + [7] * 60
    c = Q8Cache(lens, 4, 128, 64, fmt)
    g = torch.Generator().manual_seed(2)
    check_append(c, q, torch.randn(sum(q), 4, 128, generator=g).to(BF16), torch.randn(sum(q), 4, 128, generator=g).to(BF16))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_append_off_the_vector_boundaries(fmt, dtype):
    c = Q8Cache([9], 2, 64, 16, fmt)
    g = torch.Generator().manual_seed(3)
    x = torch.randn(9, 2, 66, generator=g).to(dtype)
    gx = x.cuda()
    check_append(c, [9], x[..., 1:65], x[..., 2:], gx[..., 1:65], gx[..., 2:])


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_append_values_at_the_limits(fmt, dtype):
    """Zeros, the smallest and largest numbers, halves between codes, and vectors that are not finite."""
    info = torch.finfo(dtype)
    x = torch.zeros(12, 1, 64)
    x[1, 0, 3] = info.smallest_normal
    x[2, 0, 7] = -info.max
    x[3] = info.max
    x[4, 0, :5] = torch.tensor([254.0, 1.0, 3.0, -1.0, -3.0])        # int8: 127 and halves
    x[5, 0, :6] = torch.tensor([448.0, 17.0, 19.0, -21.0, 0.0009765625, 0.0029296875])  # e4m3: ties
    x[6, 0, 1] = float("nan")
    x[7, 0, 63] = float("inf")
    x[8, 0, 0], x[8, 0, 1] = float("-inf"), float("nan")
    x[9, 0, 5] = 2.0 ** -133 if dtype == BF16 else 2.0 ** -24        # the smallest subnormal
    x[10, 0, :2] = torch.tensor([-0.0, 0.0])
    x[11, 0, :3] = torch.tensor([1.0, 2.0 ** -12, -2.0 ** -9])
    x = x.to(dtype)
    c = Q8Cache([12], 1, 64, 16, fmt)
    check_append(c, [12], x, x.flip(0))
    for t in (6, 7, 8):
        page = int(c.table[0, 0])
        assert torch.isnan(c.gks[page, t, 0]) and not raw(c.gkc)[page, t].any()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_append_negative_zeros_and_what_rounds_to_them(fmt, dtype):
    x = torch.randn(16, 2, 64, generator=torch.Generator().manual_seed(6))
    x[:, :, ::3] = -0.0
    x[:, :, 1::3] *= -1e-6
    check_append(Q8Cache([16], 2, 64, 16, fmt), [16], x.to(dtype), x.flip(0).to(dtype))


def test_append_bad_pages_lengths_and_rows():
    """Each is skipped and told; the others are written."""
    for what in ("page", "negative page", "length", "order", "none"):
        c = Q8Cache([20, 20, 20], 2, 64, 16, E4M3)
        cu, table, kv_len = torch.tensor([1, 3, 5, 7], dtype=torch.int32), c.table.clone(), c.kv_len.cpu().clone()
        if what == "page":
            table[1, 1] = c.pages
        if what == "negative page":
            table[1, 1] = -1
        if what == "length":
            kv_len[1] = 33
        if what == "order":
            cu[2] = 9
        x = torch.randn(8, 2, 64).to(BF16)
        gx = x.cuda()
        ws = new_ws()
        moe.moe_kv_append_q8(gx, gx, c.gkc, c.gvc, c.gks, c.gvs, table.cuda(), cu.cuda(), kv_len.cuda(), ws)
        assert status(ws) == (0 if what == "none" else moe.MOE_ERR_DEVICE_BOUNDS)
        q, d = quantise(x, E4M3)
        want = raw(c.kc).clone()
        for b in (0, 1, 2):
            if what == "order" and b or b == 1 and what != "none":
                continue
            for i in (0, 1):
                want[int(c.table[b, 1]), 2 + i] = raw(q)[1 + 2 * b + i]
        assert torch.equal(raw(c.gkc).cpu(), want), what


# ------------------------------------------------------------------ reading back

def check_read(c, first, rows, dtype, gaps=False):
    ko = torch.full((rows, c.Hkv + gaps, c.D + 8 * gaps), 7.0, dtype=dtype, device="cuda")[:, :c.Hkv, :c.D]
    vo = torch.full((rows, c.Hkv, c.D), 7.0, dtype=dtype, device="cuda")
    ws = new_ws()
    moe.moe_kv_read_q8(c.gkc, c.gvc, c.gks, c.gvs, c.gtable, c.kv_len, torch.tensor(first, dtype=torch.int32).cuda(), ko,
                       vo, ws)
    assert status(ws) == 0
    for name, out in (("k", ko), ("v", vo)):
        want = torch.full((rows, c.Hkv, c.D), 7.0, dtype=dtype)
        for b, n in enumerate(c.lens):
            # a product of an 8-bit code and an fp32 scale, rounded to fp32 and then to the output's type
            want[first[b]:first[b] + n] = c.sequence(b, name).float().to(dtype)
        assert torch.equal(torch.nan_to_num(out.cpu().float(), nan=-9.0), torch.nan_to_num(want.float(), nan=-9.0))


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F16, F32])
@pytest.mark.parametrize("Hkv,D,page", [(8, 128, 16), (1, 256, 64), (3, 64, 48), (2, 80, 1), (5, 8, 7)])
def test_read(fmt, dtype, Hkv, D, page):
    lens = [37, 0, 1, 130, 16]
    first = [2, 39, 41, 42, 180]
    for layout in ("rows", "heads", "odd"):
        c = Q8Cache(lens, Hkv, D, page, fmt, seed=D + 1, layout=layout)
        check_read(c, first, 200, dtype, gaps=layout == "heads")


@pytest.mark.parametrize("fmt", FMTS)
def test_read_every_code(fmt):
    """All 256 codes, and scales that are 0, NaN, tiny and large."""
    c = Q8Cache([16], 1, 256, 16, fmt)
    page = int(c.table[0, 0])
    every = torch.arange(256).to(torch.uint8)
    for t, d in enumerate([1.0, 0.0, float("nan"), 2.0 ** -126, 2.0 ** 100, 0.3]):
        for codes, gcodes, scales, gscales in ((c.kc, c.gkc, c.ks, c.gks), (c.vc, c.gvc, c.vs, c.gvs)):
            codes.view(torch.uint8)[page, t, 0] = every
            scales[page, t, 0] = d
            gcodes.copy_(codes) if fmt == INT8 else raw(gcodes).copy_(raw(codes))
            gscales.copy_(scales)
    check_read(c, [0], 16, F32)
    check_read(c, [0], 16, BF16)


def test_read_what_does_not_fit_is_told():
    c = Q8Cache([20, 20], 2, 64, 16, E4M3)
    for what, first, rows, table in [("rows", [0, 20], 39, None), ("overlap", [0, 19], 60, None),
                                     ("negative", [-1, 30], 60, None), ("page", [0, 20], 60, (1, 1)),
                                     ("length", [0, 20], 60, None), ("fits", [0, 20], 40, None)]:
        t, kv_len = c.table.clone(), c.kv_len.clone()
        if table:
            t[table] = -5
        if what == "length":
            kv_len[1] = 33
        ko = torch.full((rows, 2, 64), 7.0, dtype=BF16, device="cuda")
        vo, ws = ko.clone(), new_ws()
        moe.moe_kv_read_q8(c.gkc, c.gvc, c.gks, c.gvs, t.cuda(), kv_len, torch.tensor(first, dtype=torch.int32).cuda(),
                           ko, vo, ws)
        assert status(ws) == (0 if what == "fits" else moe.MOE_ERR_DEVICE_BOUNDS), what
        n = 19 if what in ("overlap", "negative") else 20
        lo = 1 if what == "negative" else 0
        assert torch.equal(ko[:n].cpu(), c.sequence(0, "k").to(BF16)[lo:lo + n]), what


def test_written_then_read_back():
    """A round trip is off by half a step of the code at most: 2^-4 relative or half a subnormal step of e4m3."""
    g = torch.Generator().manual_seed(5)
    x = torch.randn(50, 4, 128, generator=g).to(BF16)
    for fmt in FMTS:
        c = Q8Cache([50], 4, 128, 16, fmt)
        cu = torch.tensor([0, 50], dtype=torch.int32).cuda()
        ws, ko = new_ws(), torch.empty(50, 4, 128, device="cuda")
        vo = torch.empty_like(ko)
        moe.moe_kv_append_q8(x.cuda(), x.cuda(), c.gkc, c.gvc, c.gks, c.gvs, c.gtable, cu, c.kv_len, ws)
        moe.moe_kv_read_q8(c.gkc, c.gvc, c.gks, c.gvs, c.gtable, c.kv_len, cu[:1], ko, vo, ws)
        d = x.float().abs().amax(-1, keepdim=True) / (448.0 if fmt == E4M3 else 127.0)
        half = torch.maximum(x.float().abs() * 2.0 ** -4, d * 2.0 ** -10) if fmt == E4M3 else d / 2
        # the quotient, the scale and the product each round once to fp32
        assert ((ko.cpu() - x.float()).abs() <= half * (1 + 2.0 ** -10) + x.float().abs() * 3 * 2.0 ** -24).all()
        assert torch.equal(ko, vo)


def test_a_captured_step_is_replayed():
    c = Q8Cache([33, 70], 2, 64, 16, E4M3)
    cu = torch.tensor([0, 1, 3], dtype=torch.int32).cuda()
    x = torch.zeros(3, 2, 64, dtype=BF16, device="cuda")
    ws, ko = new_ws(), torch.zeros(120, 2, 64, dtype=BF16, device="cuda")
    vo, first = torch.zeros_like(ko), torch.tensor([0, 40], dtype=torch.int32).cuda()

    def step():
        moe.moe_kv_append_q8(x, x, c.gkc, c.gvc, c.gks, c.gvs, c.gtable, cu, c.kv_len, ws)
        moe.moe_kv_read_q8(c.gkc, c.gvc, c.gks, c.gvs, c.gtable, c.kv_len, first, ko, vo, ws)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in (1, 2):
        x.copy_(torch.randn(3, 2, 64, generator=torch.Generator().manual_seed(seed)).to(BF16))
        graph.replay()
        q, d = quantise(x.cpu(), E4M3)
        want = (code_values(q) * d.double().unsqueeze(-1)).float().to(BF16)
        assert torch.equal(ko[[32, 108, 109]].cpu(), want) and status(ws) == 0
