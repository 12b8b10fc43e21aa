"""Attention over an 8-bit paged cache against a plain 64-bit form, within derived bounds."""
import pytest
import torch

import block_quantized_routed_gb300 as moe
from tests.q8_ref import E4M3, INT8, Q8Cache, attention, new_ws, status

pytestmark = pytest.mark.gpu
BF16, F16 = torch.bfloat16, torch.float16
FMTS = [E4M3, INT8]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe.load()


def workspace(Hq, c):
    return new_ws(moe.moe_paged_attention_q8_workspace_size(Hq, c.Hkv, c.D))


def rnd(*shape, dtype=BF16, seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def attend(c, q, q_lens, scale=None, window=0, ws=None, want=0):
    """out [T, Hq, D] and lse on the CPU; rows behind the last sequence have to stay as they were."""
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    ws = workspace(Hq, c) if ws is None else ws
    cu = torch.tensor([0] + list(q_lens)).cumsum(0).int().cuda()
    spare = 2
    gq = torch.zeros(T + spare, Hq + 1, D, dtype=q.dtype, device="cuda")
    gq[:T, :Hq] = q.cuda()
    out = torch.full((T + spare, Hq, D + 8), 7.0, dtype=q.dtype, device="cuda")
    lse = torch.full((T + spare, Hq), 7.0, device="cuda")
    moe.moe_paged_attention_q8(gq[:, :Hq], c.gkc, c.gvc, c.gks, c.gvs, c.gtable, cu, c.kv_len, scale, out[..., :D], ws,
                               lse=lse, window=window)
    assert status(ws) == want
    assert (out[T:] == 7).all() and (out[..., D:] == 7).all() and (lse[T:] == 7).all()
    assert not ws[16:1024].any()       # counters are left at zero
    return out[:T, :, :D].double().cpu(), lse[:T].double().cpu()


def check(c, q_lens, Hq, dtype=BF16, scale=None, window=0, seed=0, q=None):
    q = rnd(sum(q_lens), Hq, c.D, dtype=dtype, seed=seed) if q is None else q
    got, lse = attend(c, q, q_lens, scale, window)
    ref, ref_lse, tol, lse_tol = attention(q, c, q_lens, c.D ** -0.5 if scale is None else scale, window)
    nan = torch.isnan(ref)
    assert torch.equal(nan, torch.isnan(got)) and torch.equal(torch.isnan(ref_lse), torch.isnan(lse))
    bad = ((got - ref).abs() > tol) & ~nan
    if dtype == F16:  # numbers from 65520 on round to infinity
        bad &= ~((ref.abs() + tol >= 65520) & torch.isinf(got) & (got.sign() == ref.sign()))
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()}: {(got - ref).abs()[bad].max():.3e} beyond {tol[bad].min():.3e}"
    empty = ref_lse == -float("inf")
    assert torch.equal(lse == -float("inf"), empty) and (got[empty] == 0).all()
    assert ((lse - ref_lse).abs() <= lse_tol)[~empty & ~torch.isnan(ref_lse)].all()


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("D,Hkv,G,page", [(128, 2, 8, 16), (64, 8, 5, 32), (256, 2, 8, 16), (128, 1, 1, 64), (128, 4, 16, 48),
                                          (64, 1, 3, 256), (256, 1, 16, 64), (80, 2, 4, 16), (8, 3, 2, 16), (128, 2, 4, 7),
                                          (64, 2, 64, 16), (248, 1, 2, 1)])
def test_single_tokens_and_windows(fmt, dtype, D, Hkv, G, page):
    lens = [1, 2, 15, 16, 17, 100, 333]
    c = Q8Cache(lens, Hkv, D, page, fmt, seed=D + G)
    check(c, [1] * 7, Hkv * G, dtype)
    check(c, [1, 2, 4, 0, 16, 3, 7], Hkv * G, dtype, seed=1)
    check(c, [1, 2, 4, 1, 16, 3, 7], Hkv * G, dtype, window=5, seed=2)


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("layout", ["heads", "rows"])
def test_layouts_of_the_cache(fmt, layout):
    c = Q8Cache([70, 1, 40], 3, 128, 32, fmt, layout=layout)
    check(c, [1, 1, 5], 6, BF16)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("kv", [1000, 4097, 20000])
def test_long_pasts_shared_by_many_ctas(D, kv):
    """Items that many CTAs share and join, alone and beside short ones."""
    c = Q8Cache([kv], 1, D, 16, E4M3, seed=kv)
    check(c, [1], 8)
    check(c, [3], 4, seed=1)
    c = Q8Cache([5, kv, 17, kv // 2, 1], 2, D, 64, INT8, seed=kv)
    check(c, [1, 1, 1, 1, 1], 16, F16)
    check(c, [4, 2, 9, 1, 1], 6, BF16, window=kv // 3)


def test_many_sequences_of_all_lengths():
    g = torch.Generator().manual_seed(7)
    lens = torch.randint(1, 600, (130,), generator=g).tolist()
    c = Q8Cache(lens, 2, 64, 16, E4M3)
    check(c, [1] * 130, 8)
    check(c, [min(n, 1 + i % 5) for i, n in enumerate(lens)], 4, F16, window=100)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_chunks_of_many_tokens(D):
    c = Q8Cache([150, 33], 2, D, 16, E4M3)
    check(c, [120, 33], 10)
    check(c, [120, 33], 6, window=20, seed=1)


def test_more_new_tokens_than_keys():
    """Tokens that stand before the first key see nothing: zeros, and lse of -inf."""
    c = Q8Cache([3, 0, 40], 2, 128, 16, INT8)
    q = rnd(5 + 2 + 1, 8, 128)
    got, lse = attend(c, q, [5, 2, 1])
    assert (got[:2] == 0).all() and (lse[:2] == -float("inf")).all()
    assert (got[5:7] == 0).all() and (lse[5:7] == -float("inf")).all()
    part = Q8Cache([3, 0, 40], 2, 128, 16, INT8)
    ref, ref_lse, tol, _ = attention(q[2:], part, [3, 2, 1], 128 ** -0.5, 0)
    assert ((got[2:] - ref).abs() <= tol).all()


@pytest.mark.parametrize("scale", [0.0, -0.3, 5.0])
def test_scales_of_the_scores(scale):
    c = Q8Cache([300, 31], 2, 128, 16, E4M3)
    check(c, [2, 1], 8, scale=scale)


@pytest.mark.parametrize("D", [64, 128, 80])
def test_magnitudes_far_apart(D):
    """Values and keys whose scales spread over many orders, a first key of zeros with most of the weight, large and
    tiny queries: the reference of the weights follows weight times scale."""
    c = Q8Cache([200, 64], 1, D, 16, E4M3, seed=3)
    g = torch.Generator().manual_seed(4)
    c.vs.mul_(torch.pow(10.0, 12 * torch.rand(c.vs.shape, generator=g) - 8))
    p0 = int(c.table[0, 0])
    c.vs[p0, 0] = 0.0                      # no values at all
    c.ks[p0, 0] *= 30.0
    c.vs[p0, 1] = 2.0 ** -126
    c.ks[p0, 2] = 0.0
    for t, gt in ((c.ks, c.gks), (c.vs, c.gvs)):
        gt.copy_(t)
    for size in (1e-20, 1.0, 1e4):
        check(c, [2, 1], 8, BF16, scale=0.05 / min(size, 1.0) if size < 1 else 0.05 / size, q=(rnd(3, 8, D).float() * size).to(BF16))
    q = rnd(3, 8, D).float()
    q[..., ::3] *= 1e-6                    # elements far below the row's largest
    q[1] = 0.0
    check(c, [2, 1], 8, F16, q=q.to(F16))
    check(c, [2, 1], 8, BF16, q=q.to(BF16))


@pytest.mark.parametrize("D,page", [(128, 16), (64, 48), (80, 16)])
def test_what_is_hidden_has_no_effect(D, page):
    """NaN scales and any codes beyond the sequence, below the window, of later tokens, in pages of nobody."""
    for fmt in FMTS:
        c = Q8Cache([50, 20], 2, D, page, fmt, spare=4)
        q = rnd(4, 8, D)
        want = attend(c, q, [3, 1], window=9)
        for b, n in enumerate(c.lens):
            for pos in range(0, c.table.shape[1] * page):
                inside = n - (3 if b == 0 else 1) - 8 <= pos < n
                if not inside and pos // page < -(-n // page):
                    pg = int(c.table[b, pos // page])
                    for codes, sc in ((c.gkc, c.gks), (c.gvc, c.gvs)):
                        codes.view(torch.uint8)[pg, pos % page] = 0x7f
                        sc[pg, pos % page] = float("nan") if pos % 2 else float("inf")
        got = attend(c, q, [3, 1], window=9)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("D", [128, 80])
def test_numbers_that_are_not_finite(D):
    """A NaN scale of a key or of a value reaches the rows that see it, and no others."""
    for which in ("ks", "vs"):
        c = Q8Cache([40, 30], 2, D, 16, E4M3)
        pg = int(c.table[0, 38 // 16])
        for t in (getattr(c, which), getattr(c, "g" + which)):
            t[pg, 38 % 16, 1] = float("nan")
        q = rnd(4, 4, D)
        got, lse = attend(c, q, [3, 1])
        hit = torch.zeros(4, 4, dtype=torch.bool)
        hit[1:3, 2:] = True                    # tokens at 38 and 39, heads of key/value head 1
        assert torch.equal(torch.isnan(got).all(-1), hit) and torch.equal(torch.isnan(got).any(-1), hit)
        assert torch.equal(torch.isnan(lse), hit if which == "ks" else torch.zeros_like(hit))
    c = Q8Cache([20], 1, D, 16, E4M3)
    q = rnd(1, 4, D)
    q[0, 2, 5] = float("nan")
    got, lse = attend(c, q, [1])
    assert torch.equal(torch.isnan(got).all(-1)[0], torch.tensor([False, False, True, False]))
    assert torch.equal(torch.isnan(lse)[0], torch.tensor([False, False, True, False])) and not torch.isnan(got[0, :2]).any()


@pytest.mark.parametrize("D,Hkv", [(128, 2), (64, 1), (256, 1), (80, 2)])
@pytest.mark.parametrize("pos", [10, 37, 39])
def test_codes_that_are_nan(D, Hkv, pos):
    """e4m3's NaN in a key or a value: the rows that see it, and no others, whether all rows of a tile do or some."""
    for name in ("kc", "vc"):
        c = Q8Cache([40, 30], Hkv, D, 16, E4M3)
        q = rnd(5, 4, D)
        want, want_lse = attend(c, q, [4, 1])
        getattr(c, "g" + name).view(torch.uint8)[int(c.table[0, pos // 16]), pos % 16, Hkv - 1, 11] = 0xff
        got, lse = attend(c, q, [4, 1])
        hit = torch.zeros(5, 4, dtype=torch.bool)
        hit[max(0, pos - 36):4, 4 - 4 // Hkv:] = True
        if name == "kc":
            assert torch.isnan(got[hit]).all() and torch.isnan(lse[hit]).all()
        else:
            assert torch.isnan(got[hit][:, 11]).all() and torch.equal(lse, want_lse)
        assert torch.equal(got[~hit], want[~hit]) and torch.equal(lse[~hit], want_lse[~hit])


@pytest.mark.parametrize("D,page", [(128, 16), (80, 16)])
def test_bad_numbers_are_skipped_and_told(D, page):
    c = Q8Cache([40, 40, 40], 2, D, page, E4M3)
    q = rnd(3, 4, D)
    good, _ = attend(c, q, [1, 1, 1])
    bad = moe.MOE_ERR_DEVICE_BOUNDS
    for which in ("length", "negative"):
        ws, out = workspace(4, c), torch.full((3, 4, D), 7.0, dtype=BF16, device="cuda")
        kv_len = torch.tensor([40, 10 ** 6 if which == "length" else -1, 40], dtype=torch.int32).cuda()
        cu = torch.arange(4, dtype=torch.int32).cuda()
        moe.moe_paged_attention_q8(q.cuda(), c.gkc, c.gvc, c.gks, c.gvs, c.gtable, cu, kv_len, D ** -0.5, out, ws)
        assert status(ws) == bad
        assert torch.equal(out[[0, 2]].double().cpu(), good[[0, 2]]) and (out[1] == 7).all()
    for cu in ([0, 5, 2, 3], [0, -1, 2, 3], [2, 1, 0, 3], [0, 3, 1, 3], [0, 3, 0, 3]):
        ws, out = workspace(4, c), torch.full((3, 4, D), 7.0, dtype=BF16, device="cuda")
        moe.moe_paged_attention_q8(q.cuda(), c.gkc, c.gvc, c.gks, c.gvs, c.gtable, torch.tensor(cu, dtype=torch.int32).cuda(),
                                   c.kv_len, D ** -0.5, out, ws)
        assert status(ws) == bad
        assert not ws[16:1024].any()
    # a bad page's keys read as zeros
    c.table[1, 1] = c.gtable[1, 1] = c.pages + 3
    got, _ = attend(c, q, [1, 1, 1], want=bad)
    c.table[1, 1] = 0
    keep = c.kc.view(torch.uint8).clone(), c.vc.view(torch.uint8).clone()
    ids = c.table[1, :3].long()
    k, v = c.sequence(1, "k"), c.sequence(1, "v")
    k[16:32] = v[16:32] = 0
    a = torch.einsum("hd,jhd->hj", q[1].double(), k.repeat_interleave(2, 1)) * D ** -0.5
    ref = torch.einsum("hj,jhd->hd", torch.softmax(a, 1), v.repeat_interleave(2, 1))
    assert keep and len(ids) == 3
    assert ((got[1] - ref).abs() <= 2.0 ** -7 * ref.abs().amax()).all()
    assert torch.equal(got[[0, 2]], good[[0, 2]])


def test_results_do_not_depend_on_timing():
    c = Q8Cache([9000, 300, 4000], 2, 128, 64, E4M3)
    q = rnd(6, 16, 128)
    ws = workspace(16, c)
    want = attend(c, q, [4, 1, 1], ws=ws)
    for _ in range(5):
        got = attend(c, q, [4, 1, 1], ws=ws)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_workspaces_on_two_streams():
    c = Q8Cache([9000, 300], 2, 128, 64, E4M3)
    q = rnd(2, 16, 128).cuda()
    cu = torch.arange(3, dtype=torch.int32).cuda()
    outs = [torch.empty_like(q) for _ in range(3)]
    wss = [workspace(16, c) for _ in range(3)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(10):
        for s, out, ws in zip(streams, outs, wss):
            moe.moe_paged_attention_q8(q, c.gkc, c.gvc, c.gks, c.gvs, c.gtable, cu, c.kv_len, 0.1, out, ws, stream=s)
    torch.cuda.synchronize()
    moe.moe_paged_attention_q8(q, c.gkc, c.gvc, c.gks, c.gvs, c.gtable, cu, c.kv_len, 0.1, outs[2], wss[2])
    assert torch.equal(outs[0], outs[2]) and torch.equal(outs[1], outs[2])
    assert [status(ws) for ws in wss] == [0, 0, 0]


def test_a_captured_call_follows_the_lengths():
    """Lengths, tables and queries come from device memory at each replay."""
    c = Q8Cache([2000, 100], 2, 128, 16, INT8)
    q = rnd(2, 8, 128).cuda()
    out, lse, ws = torch.empty_like(q), torch.empty(2, 8, device="cuda"), workspace(8, c)
    cu = torch.arange(3, dtype=torch.int32).cuda()

    def step():
        moe.moe_paged_attention_q8(q, c.gkc, c.gvc, c.gks, c.gvs, c.gtable, cu, c.kv_len, 0.1, out, ws, lse=lse)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for lens in ([2000, 100], [17, 99], [1, 1], [1500, 3]):
        c.lens = lens
        c.kv_len.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        ref, ref_lse, tol, _ = attention(q.cpu(), c, [1, 1], 0.1, 0)
        assert ((out.double().cpu() - ref).abs() <= tol).all() and status(ws) == 0


def test_cache_offsets_beyond_32_bits():
    """A cache of more than 2^32 bytes: its last page is written, read and attended to."""
    page, Hkv, D = 256, 8, 256
    pages = (1 << 32) // (page * Hkv * D) + 3
    kc = torch.empty(pages, page, Hkv, D, dtype=torch.uint8, device="cuda").view(E4M3)
    ks = torch.empty(pages, Hkv, page, device="cuda").transpose(1, 2)
    c = Q8Cache([40], Hkv, D, page, E4M3, spare=0)
    table = torch.tensor([[pages - 1]], dtype=torch.int32).cuda()
    kv_len, cu = torch.tensor([40], dtype=torch.int32).cuda(), torch.tensor([0, 40], dtype=torch.int32).cuda()
    x = rnd(40, Hkv, D).cuda()
    ws = new_ws()
    moe.moe_kv_append_q8(x, x, kc, kc, ks, ks, table, cu, kv_len, ws)
    small = [torch.zeros(1, page, Hkv, D, dtype=torch.uint8, device="cuda").view(E4M3), torch.zeros(1, page, Hkv, device="cuda")]
    moe.moe_kv_append_q8(x, x, small[0], small[0], small[1], small[1], torch.zeros_like(table), cu, kv_len, ws)
    assert torch.equal(kc.view(torch.uint8)[-1, :40], small[0].view(torch.uint8)[0, :40])
    q = rnd(1, 16, D).cuda()
    outs = [torch.empty_like(q) for _ in range(2)]
    cu = torch.tensor([0, 1], dtype=torch.int32).cuda()
    for out, k8, sc, t in ((outs[0], kc, ks, table), (outs[1], small[0], small[1], torch.zeros_like(table))):
        moe.moe_paged_attention_q8(q, k8, k8, sc, sc, t, cu, kv_len, 0.1, out, workspace(16, c))
    assert torch.equal(outs[0], outs[1])
    rows = [torch.empty(40, Hkv, D, device="cuda") for _ in range(2)]
    for r, k8, sc, t in ((rows[0], kc, ks, table), (rows[1], small[0], small[1], torch.zeros_like(table))):
        moe.moe_kv_read_q8(k8, k8, sc, sc, t, kv_len, cu[:1], r, torch.empty_like(r), ws)
    assert torch.equal(rows[0], rows[1]) and status(ws) == 0
