"""The decoder-block operators on the GPU against plain 64-bit forms (tests/block_ref.py).

Tolerances are derived: fp32 arithmetic to a counted number of roundings, plus half a step of each rounding to
a narrower type.  Selections, copies and codes' consistency are compared exactly."""
import numpy as np
import pytest
import torch

import block_quantized_routed_gb300 as moe
from tests import block_ref
from tests.block_ref import HALF_STEP, TINY, U32

pytestmark = pytest.mark.gpu
F32, BF16, F16 = torch.float32, torch.bfloat16, torch.float16
NAN = float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe.load()


def rnd(shape, seed, dtype=F32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype)


def status(ws):
    return moe.moe_get_status(ws)


# ------------------------------------------------------------------ norm

FMTS = {"q8k": (moe.NORM_Q_Q8K, 256, 127.0), "g128": (moe.NORM_Q_E4M3_G128, 128, 448.0),
        "e4m3": (moe.NORM_Q_E4M3_ROW, 0, 448.0), "int8": (moe.NORM_Q_INT8_ROW, 0, 127.0)}
# roundings of z: the sum of squares (a thread's 32 products, two 5-step shuffles, one more), the mean, eps,
# square root, division, two products, weight offset; half of the first group's weight through the square root
Z_REL = (32 + 11 + 8) * U32


def check_norm(x, res, w, eps, offset, s_got, y, q, d, bs, fmt):
    s, z = block_ref.norm(x, res, w, eps, offset)
    zt = z.abs() * Z_REL + s.abs() * U32 * (w.double().abs() + abs(offset)) / torch.sqrt(
        (s * s).mean(1, keepdim=True) + eps)
    if s_got is not None:
        want = x.float() if res is None else x.float() + res.float()
        assert torch.equal(s_got.cpu(), want.to(s_got.dtype))
    if y is not None:
        err = (y.cpu().double() - z).abs()
        assert (err <= 1.01 * (zt + z.abs() * HALF_STEP[y.dtype]) + TINY[y.dtype]).all()
    if fmt is None:
        return
    _, group, top = FMTS[fmt]
    T, H = z.shape
    g = group or H
    n = -(-H // g)
    pad = torch.zeros(T, n * g, dtype=torch.float64)
    pad[:, :H], zpad = z, torch.zeros(T, n * g, dtype=torch.float64)
    zpad[:, :H] = zt
    peak = pad.view(T, n, g).abs().amax(2)
    d = d.cpu().double().view(T, n)
    assert ((d - peak / top).abs() <= peak / top * (Z_REL + 4 * U32) + 2.0 ** -149).all()
    dd = d.repeat_interleave(g, 1)[:, :H]
    codes = q.cpu().float().double()
    zero = dd == 0
    assert (codes[zero] == 0).all()
    r = torch.where(zero, torch.zeros_like(z), z / torch.where(zero, torch.ones_like(dd), dd))
    rt = torch.where(zero, torch.zeros_like(z), zt / torch.where(zero, torch.ones_like(dd), dd)) + r.abs() * 4 * U32
    if top == 127.0:
        assert ((codes - r).abs() <= 0.5 + rt).all()
    else:
        assert ((codes - r).abs() <= torch.clamp(r.abs() * 2.0 ** -4, min=2.0 ** -10) * 1.001 + 1.1 * rt).all()
    if bs is not None:
        assert torch.equal(bs.cpu().double(), codes.view(T, H // 16, 16).sum(2))


@pytest.mark.parametrize("T,H", [(1, 1), (1, 2048), (3, 7), (5, 129), (37, 6144), (700, 640), (2, 16384), (400, 8192),
                                 (1000, 33), (1300, 2048), (1217, 12288), (1500, 5000)])
@pytest.mark.parametrize("xt,rt", [(BF16, None), (BF16, BF16), (BF16, F32), (F16, F16), (F16, F32), (F32, F32)])
def test_norm_types_and_sizes(T, H, xt, rt):
    x, w = rnd((T, H), 1, xt), 1 + 0.2 * rnd((H,), 2)
    res = None if rt is None else rnd((T, H), 3, rt, 4.0)
    s = torch.empty((T, H), dtype=rt or xt, device="cuda")
    for yt in (F32, BF16, F16):
        y = torch.empty((T, H), dtype=yt, device="cuda")
        moe.moe_add_rmsnorm(x.cuda(), w.cuda(), 1e-6, residual=None if res is None else res.cuda(), sum_out=s, y=y)
        check_norm(x, res, w, 1e-6, 0.0, s, y, None, None, None, None)


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("T,H", [(1, 256), (3, 2048), (600, 4096), (2, 16384), (4, 1), (5, 200), (9, 1027),
                                 (1500, 2304), (1234, 10240)])
def test_norm_codes(fmt, T, H):
    code, group, _ = FMTS[fmt]
    if fmt == "q8k" and H % 256:
        H = 256 * -(-H // 256)
    x, res, w = rnd((T, H), 4, BF16), rnd((T, H), 5, BF16, 3.0), 0.2 * rnd((H,), 6, F16)
    if T > 2:
        x[1], res[1] = 0.0, 0.0                                        # an all-zero row
        x[2, :min(H, 128)], res[2, :min(H, 128)] = 0.0, 0.0            # an all-zero group
    q = torch.empty((T, H), dtype=torch.float8_e4m3fn if fmt in ("g128", "e4m3") else torch.int8, device="cuda")
    d = torch.empty((T, -(-H // (group or H))), device="cuda")
    bs = torch.empty((T, H // 16), dtype=torch.int16, device="cuda") if fmt == "q8k" else None
    y = torch.empty((T, H), device="cuda")
    moe.moe_add_rmsnorm(x.cuda(), w.cuda(), 1e-5, residual=res.cuda(), y=y, q_fmt=code, q=q, d=d, bsum16=bs,
                        weight_offset=1.0)
    check_norm(x, res, w, 1e-5, 1.0, None, y, q, d, bs, fmt)
    if fmt == "q8k":  # the same codes, bit for bit, as quantizing the normalised rows
        q2, d2, bs2 = torch.empty_like(q), torch.empty_like(d), torch.empty_like(bs)
        moe.moe_q8k_quantize(y, q2, d2, bs2)
        assert torch.equal(q, q2) and torch.equal(d, d2) and torch.equal(bs, bs2)


@pytest.mark.parametrize("fmt", list(FMTS))
@pytest.mark.parametrize("T,H", [(3, 256), (400, 1536), (5, 6400), (700, 10240)])
def test_norm_codes_of_rows_off_the_boundary(fmt, T, H):
    code, group, _ = FMTS[fmt]
    x, res, w = rnd((T, H), 7, BF16), rnd((T, H), 8, F32, 3.0), 1 + 0.2 * rnd((H,), 9)
    xb = torch.full((T, H + 3), NAN, dtype=BF16, device="cuda")
    xb[:, 1:H + 1] = x.cuda()
    q = torch.empty((T, H), dtype=torch.float8_e4m3fn if fmt in ("g128", "e4m3") else torch.int8, device="cuda")
    d = torch.empty((T, -(-H // (group or H))), device="cuda")
    bs = torch.empty((T, H // 16), dtype=torch.int16, device="cuda") if fmt == "q8k" else None
    y = torch.empty((T, H), device="cuda")
    moe.moe_add_rmsnorm(xb[:, 1:H + 1], w.cuda(), 1e-5, residual=res.cuda(), y=y, q_fmt=code, q=q, d=d, bsum16=bs)
    check_norm(x, res, w, 1e-5, 0.0, None, y, q, d, bs, fmt)
    if fmt == "q8k":
        q2, d2, bs2 = torch.empty_like(q), torch.empty_like(d), torch.empty_like(bs)
        moe.moe_q8k_quantize(y, q2, d2, bs2)
        assert torch.equal(q, q2) and torch.equal(d, d2) and torch.equal(bs, bs2)


@pytest.mark.parametrize("H,off,stride", [(512, 0, 640), (512, 1, 640), (512, 0, 643), (100, 3, 131)])
def test_norm_strides_and_alignment(H, off, stride):
    T = 5
    x, res, w = rnd((T, H), 7, BF16), rnd((T, H), 8), 1 + 0.1 * rnd((H,), 9, BF16)
    xb = torch.full((T, stride), NAN, dtype=BF16, device="cuda")
    rb, sb = torch.full((T, stride), NAN, device="cuda"), torch.full((T, stride), 7.0, device="cuda")
    yb = torch.full((T, stride), 7.0, dtype=F16, device="cuda")
    cut = lambda t: t[:, off:off + H]
    cut(xb).copy_(x), cut(rb).copy_(res)
    moe.moe_add_rmsnorm(cut(xb), w.cuda(), 1e-6, residual=cut(rb), sum_out=cut(sb), y=cut(yb))
    check_norm(x, res, w, 1e-6, 0.0, cut(sb), cut(yb), None, None, None, None)
    for t in (sb, yb):                                                  # nothing written outside
        assert (t[:, :off] == 7).all() and (t[:, off + H:] == 7).all()


def test_norm_in_place_and_bad_rows():
    x, w = rnd((4, 512), 10, BF16), torch.ones(512)
    res = rnd((4, 512), 11, BF16)
    bad = x.clone()
    bad[2, 5] = NAN
    bad[3, 9] = float("inf")
    r = res.cuda()
    y = torch.empty((4, 512), device="cuda")
    q, d = torch.empty((4, 512), dtype=torch.int8, device="cuda"), torch.empty((4, 2), device="cuda")
    moe.moe_add_rmsnorm(bad.cuda(), w.cuda(), 1e-6, residual=r, sum_out=r, y=y, q_fmt=moe.NORM_Q_Q8K, q=q, d=d)
    check_norm(x[:2], res[:2], w, 1e-6, 0.0, r[:2], y[:2], q[:2], d[:2], None, "q8k")


# ------------------------------------------------------------------ routing

def check_route(l, bias, k, sigmoid=True, n_group=1, topk_group=1, top2=True, renorm=True, scale=1.0, dtype=F32):
    lt = torch.from_numpy(l).to(dtype)
    T = l.shape[0]
    ids = torch.full((T, k), -1, dtype=torch.int32, device="cuda")
    gates = torch.full((T, k), NAN, device="cuda")
    moe.moe_route_grouped(lt.cuda(), k, ids, gates, bias=None if bias is None else torch.from_numpy(bias).cuda(),
                          route=moe.ROUTE_SIGMOID if sigmoid else moe.ROUTE_SOFTMAX, n_group=n_group,
                          topk_group=topk_group, group_score=moe.GROUP_TOP2 if top2 else moe.GROUP_MAX,
                          renorm=renorm, scale=scale)
    want, g = block_ref.route(lt.float().numpy(), bias, k, sigmoid, n_group, topk_group, top2, renorm, scale)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)
    # a score: exp within 2 ulp of an argument rounded at its size (<= 104), a sum of up to 32 + 5 terms, a
    # division; then a sum of k, a division, the scale
    tol = (4 + 104 + 37 + 4) * U32 if not sigmoid else 8 * U32
    np.testing.assert_array_less(np.abs(gates.cpu().numpy() - g), np.abs(g) * (2 * tol + 20 * U32) + 1e-38)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (3, 2, 2), (4, 512, 10), (130, 33, 5), (7, 1024, 16), (1021, 192, 8),
                                   (2500, 256, 8), (5, 1000, 3)])
@pytest.mark.parametrize("sigmoid", [True, False])
@pytest.mark.parametrize("with_bias", [True, False])
def test_route_sizes(T, E, k, sigmoid, with_bias):
    rng = np.random.default_rng(T * 7 + E)
    l = (1.5 * rng.standard_normal((T, E))).astype(np.float32)
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32) if with_bias else None
    for dtype in (F32, BF16, F16):
        check_route(l, bias, k, sigmoid, dtype=dtype, renorm=dtype != F16, scale=2.5 if dtype == BF16 else 1.0)


@pytest.mark.parametrize("E,n_group,topk_group,k", [(256, 8, 4, 8), (160, 8, 3, 6), (64, 32, 5, 10), (24, 3, 2, 7),
                                                    (512, 16, 1, 16), (12, 12, 4, 4), (1000, 5, 2, 9), (256, 8, 8, 8),
                                                    (128, 4, 2, 4), (32, 8, 2, 8)])
@pytest.mark.parametrize("top2", [True, False])
def test_route_groups(E, n_group, topk_group, k, top2):
    rng = np.random.default_rng(E + n_group)
    l = (1.5 * rng.standard_normal((301, E))).astype(np.float32)
    bias = (0.1 * rng.standard_normal(E)).astype(np.float32)
    for sigmoid in (True, False):
        check_route(l, bias, k, sigmoid, n_group, topk_group, top2)
        check_route(l, None, k, sigmoid, n_group, topk_group, top2, dtype=BF16)


@pytest.mark.parametrize("E", [65, 129, 257, 320, 384, 385, 512, 513, 600, 640, 641, 768, 769, 896])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_route_numbers_of_experts(E, sigmoid):
    """Sizes around those at which a lane's number of elements changes; groups that straddle lanes."""
    rng = np.random.default_rng(E)
    l = (1.5 * rng.standard_normal((77, E))).astype(np.float32)
    bias = (0.05 * rng.standard_normal(E)).astype(np.float32)
    for dtype in (F32, BF16, F16):
        check_route(l, bias, 16, sigmoid, dtype=dtype)
        check_route(l, None, 3, sigmoid, dtype=dtype)
    for n_group in (n for n in (2, 3, 4, 5, 7, 8, 15, 16, 31, 32) if E % n == 0):
        keep = max(1, n_group // 3)
        for top2 in (True, False):
            check_route(l, bias, min(6, keep * (E // n_group)), sigmoid, n_group, keep, top2)
    shifted = torch.zeros(E + 1, device="cuda")[1:]         # a bias off the 16-byte boundary
    shifted.copy_(torch.from_numpy(bias))
    ids = torch.full((77, 8), -1, dtype=torch.int32, device="cuda")
    gates = torch.full((77, 8), NAN, device="cuda")
    moe.moe_route_grouped(torch.from_numpy(l).cuda(), 8, ids, gates, bias=shifted,
                          route=moe.ROUTE_SIGMOID if sigmoid else moe.ROUTE_SOFTMAX)
    want, _ = block_ref.route(l, bias, 8, sigmoid, 1, 1, False, True, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)


def test_route_ties_go_to_the_lower_index():
    l = np.tile(np.array([1.0, 1.0, 0.5, 1.0, -2.0, 0.5], np.float32), (40, 16))          # 96 experts, many equal
    for bias in (None, np.zeros(96, np.float32)):
        for sigmoid in (True, False):
            check_route(l, bias, 12, sigmoid)
            check_route(l, bias, 12, sigmoid, n_group=16, topk_group=3)


def test_route_keys_closer_than_fp32():
    """Keys that differ by less than fp32 rounding are still ordered as 64-bit keys are."""
    rng = np.random.default_rng(3)
    T, E = 64, 64
    l = rng.uniform(-1, 1, (T, E)).astype(np.float32)
    bias = rng.uniform(0, 0.1, E).astype(np.float32)
    for t in range(T):                      # several experts' keys within 1e-9 .. 1e-7 of one target
        target = 0.9 + 0.01 * rng.random()
        for e in rng.permutation(E)[:12]:
            p = target - float(bias[e])
            l[t, e] = np.float32(np.log(p / (1 - p)))
    check_route(l, bias, 8)
    check_route(l, bias, 8, n_group=4, topk_group=2)
    check_route(l, bias, 8, n_group=4, topk_group=2, top2=False)


@pytest.mark.parametrize("E,n_group,topk_group", [(256, 1, 1), (1024, 1, 1), (256, 8, 3), (90, 5, 2)])
def test_route_whole_rows_closer_than_fp32(E, n_group, topk_group):
    """Every expert's key within fp32 rounding of every other's: more candidates than fit a warp."""
    rng = np.random.default_rng(E + n_group)
    bias = rng.uniform(0, 0.2, E).astype(np.float32)
    l = np.empty((6, E), np.float32)
    for t in range(6):
        p = 0.7 - bias.astype(np.float64) + rng.uniform(-1, 1, E) * 1e-8
        l[t] = np.log(p / (1 - p)).astype(np.float32)
    check_route(l, bias, 8, True, n_group, topk_group)
    check_route(l, bias, 8, True, n_group, topk_group, top2=False)
    # softmax: equal logits but for the last bits, and a bias that undoes what they differ by
    l = (1.0 + rng.integers(0, 3, (6, E)) * 2.0 ** -23).astype(np.float32)
    check_route(l, (rng.integers(0, 3, E) * 1e-10).astype(np.float32), 8, False, n_group, topk_group)


def test_route_masked_and_special_logits():
    rng = np.random.default_rng(4)
    l = rng.standard_normal((9, 64)).astype(np.float32)
    l[0] = -np.inf                                          # nothing left
    l[1, 5:] = -np.inf                                      # fewer than k left
    l[2, ::2] = np.finfo(np.float32).min                    # masks of the type's lowest value
    l[3, 7] = np.nan
    l[4] = np.nan
    l[5, 3] = l[5, 40] = np.inf
    l[6] = 0.0
    l[6, 9] = -0.0
    l[7] *= 60.0                                            # far apart scores
    bias = (0.05 * rng.standard_normal(64)).astype(np.float32)
    for sigmoid in (True, False):
        check_route(l, None, 8, sigmoid)
        check_route(l, None, 8, sigmoid, n_group=8, topk_group=2, top2=False)
        check_route(l[:7], bias, 8, sigmoid)


def test_route_rows_with_a_stride():
    l = rnd((50, 100), 12)
    wide = torch.full((50, 137), 99.0)
    wide[:, 3:103] = l
    ids, gates = torch.empty((50, 6), dtype=torch.int32, device="cuda"), torch.empty((50, 6), device="cuda")
    moe.moe_route_grouped(wide.cuda()[:, 3:103], 6, ids, gates)
    want, _ = block_ref.route(l.numpy(), None, 6, True, 1, 1, True, True, 1.0)
    np.testing.assert_array_equal(ids.cpu().numpy(), want)


# ------------------------------------------------------------------ the cache

class Cache:
    """A paged cache with every unused key and value NaN and every unused page-table entry garbage."""

    def __init__(self, q_lens, kv_lens, hkv, D, page, dtype, seed, heads_first=False, spare=3):
        self.q_lens, self.kv_lens = list(q_lens), list(kv_lens)
        need = [-(-k // page) for k in kv_lens]
        pages, most = sum(need) + spare, max(1, max(need))
        g = torch.Generator().manual_seed(seed)
        order = torch.randperm(pages, generator=g)
        shape = (pages, page, hkv, D)
        self.k, self.v = torch.full(shape, NAN, dtype=dtype), torch.full(shape, NAN, dtype=dtype)
        self.table = torch.full((len(need), most), -7, dtype=torch.int32)
        at = 0
        for b, (n, kv) in enumerate(zip(need, kv_lens)):
            ids = order[at:at + n]
            at += n
            self.table[b, :n] = ids.to(torch.int32)
            fk, fv = torch.full((n * page, hkv, D), NAN), torch.full((n * page, hkv, D), NAN)
            fk[:kv], fv[:kv] = rnd((kv, hkv, D), seed + 2 * b + 1), rnd((kv, hkv, D), seed + 2 * b + 2) + 0.3
            self.k[ids], self.v[ids] = fk.view(n, page, hkv, D).to(dtype), fv.view(n, page, hkv, D).to(dtype)
        self.table[self.table < 0] = pages + 1000000
        self.cu = torch.tensor([0] + list(np.cumsum(q_lens)), dtype=torch.int32)
        self.kv = torch.tensor(kv_lens, dtype=torch.int32)
        self.T = int(self.cu[-1])
        move = lambda t: (t.permute(0, 2, 1, 3).contiguous().cuda().permute(0, 2, 1, 3) if heads_first else t.cuda())
        self.dk, self.dv = move(self.k), move(self.v)
        self.dtable, self.dcu, self.dkv = self.table.cuda(), self.cu.cuda(), self.kv.cuda()


@pytest.mark.parametrize("q_lens,kv_lens,hkv,D,page", [
    ([1], [1], 1, 64, 16), ([3, 0, 5], [3, 7, 90], 2, 128, 32), ([1] * 70, list(range(1, 71)), 8, 128, 16),
    ([700, 33], [900, 33], 3, 24, 7), ([2, 2], [40, 2], 5, 8, 1), ([17], [300], 4, 256, 256)])
@pytest.mark.parametrize("strided,heads_first", [(False, False), (True, True)])
def test_append(q_lens, kv_lens, hkv, D, page, strided, heads_first):
    c = Cache(q_lens, kv_lens, hkv, D, page, BF16, 20, heads_first)
    new = rnd((c.T + 2, 2 * hkv + 1, D + (3 if strided else 0)), 21, BF16).cuda()
    kn, vn = new[:, :hkv, :D], new[:, hkv + 1:, :D]
    if not strided:
        kn, vn = kn.contiguous(), vn.contiguous()
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    moe.moe_kv_append(kn, vn, c.dk, c.dv, c.dtable, c.dcu, c.dkv, ws)      # two rows more than cu_q names
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        for i in range(n):
            j, t = kv - n + i, int(c.cu[b]) + i
            p = int(c.table[b, j // page])
            c.k[p, j % page], c.v[p, j % page] = kn[t].cpu(), vn[t].cpu()
    assert status(ws) == 0
    assert torch.equal(c.dk.cpu().view(torch.int16), c.k.view(torch.int16))
    assert torch.equal(c.dv.cpu().view(torch.int16), c.v.view(torch.int16))


def test_append_skips_what_is_out_of_range():
    c = Cache([2, 2, 2], [20, 20, 20], 2, 64, 16, BF16, 22)
    c.dtable[0, 1] = c.k.shape[0]                  # a page beyond the cache
    c.dkv[1] = 1                                   # two new tokens, one key: a position before the start
    kn = rnd((6, 2, 64), 23, BF16).cuda()
    ws = torch.zeros(16, dtype=torch.uint8, device="cuda")
    moe.moe_kv_append(kn, kn, c.dk, c.dv, c.dtable, c.dcu, c.dkv, ws)
    assert status(ws) == moe.MOE_ERR_DEVICE_BOUNDS
    assert status(ws) == 0                         # reading clears it
    p = c.table[1, 0]
    c.k[p, 0] = kn[3].cpu()
    p = c.table[2, 1]
    c.k[p, 2], c.k[p, 3] = kn[4].cpu(), kn[5].cpu()
    assert torch.equal(c.dk.cpu().view(torch.int16), c.k.view(torch.int16))


# ------------------------------------------------------------------ attention

def attend(c, hq, D, scale, window, dtype, seed, strided=False, ws=None, lse=True):
    q = rnd((c.T, hq + 2, D), seed, dtype)
    q = q[:, 1:1 + hq] if strided else q[:, :hq].contiguous()
    dq = q.cuda() if not strided else rnd((c.T, hq + 2, D), seed, dtype).cuda()[:, 1:1 + hq]
    pad = 8 if strided else 0                      # heads of out on 16-byte, not on 32-byte boundaries
    out = torch.full((c.T, hq + (1 if strided else 0), D + pad), 5.0, dtype=dtype, device="cuda")[:, :hq, :D]
    l = torch.full((c.T, hq), NAN, device="cuda") if lse else None
    if ws is None:
        ws = torch.zeros(moe.moe_paged_attention_workspace_size(hq, c.k.shape[2], D), dtype=torch.uint8, device="cuda")
    moe.moe_paged_attention(dq, c.dk, c.dv, c.dtable, c.dcu, c.dkv, scale, out, ws, lse=l, window=window)
    return q, out, l, ws


def check_attention(q_lens, kv_lens, hq, hkv, D, page, dtype=BF16, window=0, scale=None, **kw):
    c = Cache(q_lens, kv_lens, hkv, D, page, dtype, 30 + D, heads_first=kw.pop("heads_first", False))
    scale = D ** -0.5 if scale is None else scale
    q, out, l, ws = attend(c, hq, D, scale, window, dtype, 31, **kw)
    assert status(ws) == 0
    want, wl, tol, ltol = block_ref.attention(q, c.k, c.v, c.table, c.q_lens, c.kv_lens, scale, window, dtype)
    got = out.cpu().double()
    assert torch.isfinite(got).all()
    bad = (got - want).abs() > tol
    assert not bad.any(), f"{int(bad.sum())} elements off; worst {float(((got - want).abs() / tol).max()):.2f} tolerances"
    if l is not None:
        gl = l.cpu().double()
        none = torch.isneginf(wl)
        assert torch.equal(torch.isneginf(gl), none)
        assert ((gl - wl).abs()[~none] <= ltol[~none]).all(), float(((gl - wl).abs()[~none] / ltol[~none]).max())
    return c


GEN = [  # sizes off the tensor-core form
    ([1], [1], 1, 1, 8, 1), ([3, 1], [9, 40], 4, 2, 80, 16), ([5], [33], 6, 2, 96, 24), ([2, 0, 1], [2, 5, 130], 3, 1, 64, 10),
]


@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,D,page", GEN)
@pytest.mark.parametrize("dtype", [BF16, F16])
def test_attention_general_sizes(q_lens, kv_lens, hq, hkv, D, page, dtype):
    check_attention(q_lens, kv_lens, hq, hkv, D, page, dtype)
    check_attention(q_lens, kv_lens, hq, hkv, D, page, dtype, window=4, strided=True)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv,page", [
    ([1], [1], 1, 1, 16), ([1], [777], 16, 2, 16), ([1, 1, 1], [5, 128, 129], 8, 8, 32),
    ([4, 0, 2, 1], [4, 60, 300, 1000], 20, 4, 64), ([130], [130], 4, 2, 128), ([40, 300], [700, 300], 6, 2, 16),
    ([1] * 20, [50 * i + 1 for i in range(20)], 4, 1, 256)])
def test_attention_tensor_core_sizes(q_lens, kv_lens, hq, hkv, page, D, dtype):
    check_attention(q_lens, kv_lens, hq, hkv, D, page, dtype)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("G", [1, 2, 3, 5, 7, 8, 16, 48, 160])
def test_attention_shared_heads(G, D):
    check_attention([1, 9, 2], [200, 9, 131], G, 1, D, 32)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("window", [1, 15, 16, 100, 128, 129, 1000])
def test_attention_window(window, D):
    check_attention([1, 3, 150], [400, 513, 420], 4, 2, D, 32, window=window)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_window_frees_old_pages(D):
    """Pages that lie wholly before every window of a call are never read: their table entries may be stale."""
    window, page = 40, 16
    c = Cache([3, 1], [300, 90], 2, D, page, BF16, 40)
    ref_table = c.table.clone()
    for b in range(2):
        first = (c.kv_lens[b] - c.q_lens[b] + 1 - window) // page
        c.dtable[b, :first] = 10 ** 6
        c.dk[c.table[b, :first].long().cuda()] = NAN
        c.dv[c.table[b, :first].long().cuda()] = NAN
    q, out, l, ws = attend(c, 4, D, 0.1, window, BF16, 41)
    assert status(ws) == 0
    want, _, tol, _ = block_ref.attention(q, c.k, c.v, ref_table, c.q_lens, c.kv_lens, 0.1, window, BF16)
    assert ((out.cpu().double() - want).abs() <= tol).all()


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kw", [dict(strided=True), dict(heads_first=True), dict(lse=False), dict(scale=0.0),
                                dict(scale=-0.3), dict(scale=4.0)])
def test_attention_layouts_and_scales(D, kw):
    check_attention([2, 70], [150, 200], 6, 3, D, 32, **kw)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_rows_that_see_nothing(D):
    """More new tokens than keys: the first tokens stand before the first key."""
    check_attention([5, 3, 1, 200], [2, 0, 0, 150], 4, 2, D, 16)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_growing_scores(D):
    """Scores that rise along the sequence, so that the running maximum keeps moving."""
    c = Cache([1, 40], [1500, 900], 1, D, 64, BF16, 50)
    up = torch.linspace(0.0, 6.0, 1500)
    for b, kv in enumerate(c.kv_lens):
        for j in range(kv):
            c.k[c.table[b, j // 64], j % 64] = float(up[j] if b == 0 else up[j] * (-1) ** (j // 100))
    c.dk.copy_(c.k)
    q = torch.full((c.T, 2, D), 1.0, dtype=BF16)
    q[:, 1] = -1.0
    out = torch.empty((c.T, 2, D), dtype=BF16, device="cuda")
    lse = torch.empty((c.T, 2), device="cuda")
    ws = torch.zeros(moe.moe_paged_attention_workspace_size(2, 1, D), dtype=torch.uint8, device="cuda")
    moe.moe_paged_attention(q.cuda(), c.dk, c.dv, c.dtable, c.dcu, c.dkv, 0.25, out, ws, lse=lse)
    want, wl, tol, ltol = block_ref.attention(q, c.k, c.v, c.table, c.q_lens, c.kv_lens, 0.25, 0, BF16)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    assert ((lse.cpu().double() - wl).abs() <= ltol).all()


@pytest.mark.parametrize("D", [64, 128])
def test_attention_many_sequences(D):
    n = 600
    check_attention([i % 3 for i in range(n)], [(i * 37) % 200 + 2 for i in range(n)], 2, 1, D, 16)


def test_attention_long_chunk_and_split():
    """A prompt chunk of several row tiles, and one long sequence that many CTAs share."""
    check_attention([600], [2100], 8, 2, 128, 64)
    check_attention([1], [20000], 8, 1, 128, 64)


def test_attention_workspace_is_reused():
    """The counters are left as they were found: calls of other shapes follow on the same workspace; results do
    not depend on what it held, and are the same bits each time."""
    ws = torch.zeros(moe.moe_paged_attention_workspace_size(16, 2, 128), dtype=torch.uint8, device="cuda")
    c1 = Cache([1, 1], [3000, 50], 2, 128, 64, BF16, 60)
    c2 = Cache([300], [500], 2, 128, 16, BF16, 61)
    first = [attend(c, 16, 128, 0.1, 0, BF16, 62, ws=ws)[1].clone() for c in (c1, c2)]
    for _ in range(3):
        for c, want in zip((c1, c2), first):
            assert torch.equal(attend(c, 16, 128, 0.1, 0, BF16, 62, ws=ws)[1].view(torch.int16), want.view(torch.int16))
    assert status(ws) == 0


DIVISIONS = [  # the ways in which a call's work is divided: new tokens, keys, query heads, key/value heads
    ([1] * 90, [i * 53 % 250 + 1 for i in range(90)], 8, 4),         # whole items, several to a CTA, over 32 sequences
    ([40] * 20, [40 + 9 * i for i in range(20)], 16, 2),             # whole items of several row tiles
    ([4, 0, 4, 4], [3000, 0, 130, 4], 16, 2),                        # equal numbers; an item of fewer tiles than CTAs
    ([60], [2500], 16, 2),                                           # equal numbers, many rows
    ([1] * 40, [2000 - 25 * i for i in range(40)], 8, 1),            # equal numbers, over 32 sequences
    ([1] * 100, [i * 131 % 4000 + 500 for i in range(100)], 8, 1),   # even shares, few rows
    ([30] * 50, [1000 + 10 * i for i in range(50)], 8, 2),           # even shares, many rows
]


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv", DIVISIONS)
def test_attention_division_of_work(q_lens, kv_lens, hq, hkv, D):
    check_attention(q_lens, kv_lens, hq, hkv, D, 64)


def test_attention_divisions_share_a_workspace():
    """Calls that divide their work in different ways leave the counters as they found them."""
    ws = torch.zeros(moe.moe_paged_attention_workspace_size(16, 2, 128), dtype=torch.uint8, device="cuda")
    cs = [(Cache(q, kv, hkv, 128, 64, BF16, 90), hq) for q, kv, hq, hkv in DIVISIONS if hkv == 2]
    first = [attend(c, hq, 128, 0.1, 0, BF16, 91)[1].clone() for c, hq in cs]
    for _ in range(3):
        for (c, hq), want in zip(cs, first):
            assert torch.equal(attend(c, hq, 128, 0.1, 0, BF16, 91, ws=ws)[1].view(torch.int16), want.view(torch.int16))
    assert status(ws) == 0


@pytest.mark.parametrize("D,page", [(64, 32), (128, 16), (256, 64), (80, 16)])
def test_attention_bad_tables_are_reported(D, page):
    c = Cache([2, 3, 1], [100, 90, 70], 2, D, page, BF16, 63)
    c.dtable[1, 0] = -3                      # a page that is none: reported, its keys read as zeros
    q, out, _, ws = attend(c, 4, D, 0.1, 0, BF16, 64)
    assert status(ws) == moe.MOE_ERR_DEVICE_BOUNDS
    want, _, tol, _ = block_ref.attention(q, c.k, c.v, c.table, c.q_lens, c.kv_lens, 0.1, 0, BF16)
    good = [0, 1, 5]
    assert ((out.cpu().double() - want).abs() <= tol)[good].all()
    c.dtable[1, 0] = c.table[1, 0].cuda()
    c.dkv[1] = 1 << 20                       # more keys than the table has pages: the sequence is skipped
    q, out, _, ws = attend(c, 4, D, 0.1, 0, BF16, 64)
    assert status(ws) == moe.MOE_ERR_DEVICE_BOUNDS
    assert ((out.cpu().double() - want).abs() <= tol)[good].all() and (out[2:5] == 5).all()
    c.dkv[1] = 90
    c.dcu[3] = 1000                          # a sequence beyond q's rows
    q, out, _, ws = attend(c, 4, D, 0.1, 0, BF16, 64)
    assert status(ws) == moe.MOE_ERR_DEVICE_BOUNDS
    assert ((out.cpu().double() - want).abs() <= tol)[:5].all() and (out[5] == 5).all()


@pytest.mark.parametrize("D,page", [(128, 64), (256, 16), (80, 16)])
def test_cache_offsets_beyond_32_bits(D, page):
    """Pages whose first element lies past 2^31: appended to, then attended over."""
    hkv, hq, n, kv = 4, 8, 3, 100
    pages = (1 << 31) // (page * hkv * D) + 40
    kc = torch.empty(pages, page, hkv, D, dtype=BF16, device="cuda")
    vc = torch.empty(pages, page, hkv, D, dtype=BF16, device="cuda")
    need = -(-kv // page)
    ids = torch.arange(pages - need, pages, dtype=torch.int32)
    small_k, small_v = rnd((need, page, hkv, D), 90, BF16), rnd((need, page, hkv, D), 91, BF16)
    kc[pages - need:], vc[pages - need:] = small_k.cuda(), small_v.cuda()
    q, kn, vn = rnd((n, hq, D), 92, BF16), rnd((n, hkv, D), 93, BF16), rnd((n, hkv, D), 94, BF16)
    table, cu = ids.view(1, -1).cuda(), torch.tensor([0, n], dtype=torch.int32, device="cuda")
    lens = torch.tensor([kv], dtype=torch.int32, device="cuda")
    ws = torch.zeros(moe.moe_paged_attention_workspace_size(hq, hkv, D), dtype=torch.uint8, device="cuda")
    moe.moe_kv_append(kn.cuda(), vn.cuda(), kc, vc, table, cu, lens, ws)
    out = torch.empty(n, hq, D, dtype=BF16, device="cuda")
    moe.moe_paged_attention(q.cuda(), kc, vc, table, cu, lens, 0.1, out, ws)
    assert status(ws) == 0
    for i in range(n):
        j = kv - n + i
        small_k[j // page, j % page], small_v[j // page, j % page] = kn[i], vn[i]
    assert torch.equal(kc[pages - need:].cpu(), small_k) and torch.equal(vc[pages - need:].cpu(), small_v)
    local = torch.arange(need, dtype=torch.int32).view(1, -1)
    want, _, tol, _ = block_ref.attention(q, small_k, small_v, local, [n], [kv], 0.1, 0, BF16)
    assert ((out.cpu().double() - want).abs() <= tol).all()


# ------------------------------------------------------------------ streams and graphs

def test_other_stream_and_graph():
    """All four on a side stream, then captured into a graph and replayed on changed inputs."""
    D, hq, hkv, page = 128, 8, 2, 32
    c = Cache([1, 2], [500, 70], hkv, D, page, BF16, 70)
    x, w, res = rnd((3, 512), 71, BF16).cuda(), torch.ones(512, device="cuda"), rnd((3, 512), 72, BF16).cuda()
    q8, d = torch.empty((3, 512), dtype=torch.int8, device="cuda"), torch.empty((3, 2), device="cuda")
    s, logits = torch.empty_like(x), rnd((3, 64), 73).cuda()
    ids, gates = torch.empty((3, 4), dtype=torch.int32, device="cuda"), torch.empty((3, 4), device="cuda")
    qkv = rnd((3, hq + 2 * hkv, D), 74, BF16).cuda()
    out = torch.empty((3, hq, D), dtype=BF16, device="cuda")
    ws = torch.zeros(moe.moe_paged_attention_workspace_size(hq, hkv, D), dtype=torch.uint8, device="cuda")

    def step():
        moe.moe_add_rmsnorm(x, w, 1e-6, residual=res, sum_out=s, q_fmt=moe.NORM_Q_Q8K, q=q8, d=d)
        moe.moe_kv_append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], c.dk, c.dv, c.dtable, c.dcu, c.dkv, ws)
        moe.moe_paged_attention(qkv[:, :hq], c.dk, c.dv, c.dtable, c.dcu, c.dkv, 0.1, out, ws)
        moe.moe_route_grouped(logits, 4, ids, gates)

    def results():
        return [t.clone() for t in (s, q8, d, out, ids, gates)]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    want = results()
    step()
    assert all(torch.equal(a, b) for a, b in zip(want, results()))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    x.copy_(rnd((3, 512), 75, BF16)), qkv.copy_(rnd((3, hq + 2 * hkv, D), 76, BF16)), logits.mul_(-1)
    graph.replay()
    got = results()
    step()
    assert all(torch.equal(a, b) for a, b in zip(got, results()))
    assert not torch.equal(want[3], got[3]) and status(ws) == 0
