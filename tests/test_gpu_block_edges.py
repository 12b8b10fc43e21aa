"""The decoder-block operators where their inputs are degenerate: near-ties of unequal precision, non-finite numbers
in hidden and in visible places, underflow, limits of integers.  Plain 64-bit forms as in test_gpu_block.py."""
import numpy as np
import pytest
import torch

import block_quantized_routed_gb300 as moe
from tests import block_ref
from tests.test_gpu_block import BF16, F16, F32, Cache, attend, check_norm, check_route, rnd, status

pytestmark = pytest.mark.gpu
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _lib():
    moe.load()


# ------------------------------------------------------------------ routing: the border of the selection

def test_route_a_tie_at_the_border_hides_no_rival():
    """The k-th and the next key are the same in any precision; one further down is larger in 64 bits alone."""
    l = np.array([[17.0, 17.0, 18.0]], np.float32)
    check_route(l, np.zeros(3, np.float32), 1)
    for E, k in [(64, 3), (256, 8), (700, 8), (1024, 16)]:
        l = np.full((4, E), -5.0, np.float32)
        for t in range(4):
            l[t, 3 * t:3 * t + k + 1] = 17.0              # k + 1 equal keys, all 1 in fp32
            l[t, E - 1 - t] = 18.0
        check_route(l, np.zeros(E, np.float32), k)
        check_route(l, np.full(E, 0.25, np.float32), k)


@pytest.mark.parametrize("E,k", [(64, 4), (256, 8), (512, 10), (1024, 16)])
@pytest.mark.parametrize("sigmoid", [True, False])
def test_route_scores_of_few_values(E, k, sigmoid):
    """Logits of a narrow type repeat: saturated scores, tiny scores, whole rows of one value, more than 32 of each."""
    rng = np.random.default_rng(E + k)
    zero, half = np.zeros(E, np.float32), np.full(E, 0.5, np.float32)
    steps = rng.integers(0, 6, (24, E)).astype(np.float32) * 0.125
    for bias in (zero, half):
        check_route(17.0 + steps, bias, k, sigmoid)
        check_route(-18.0 + steps, bias, k, sigmoid)
        check_route(np.full((3, E), 2.0, np.float32), bias, k, sigmoid)
        check_route(np.where(rng.random((24, E)) < 0.5, 20.0, 19.0).astype(np.float32), bias, k, sigmoid)
        check_route(17.0 + steps, bias, min(k, 4), sigmoid, n_group=4, topk_group=2)


@pytest.mark.parametrize("E", [128, 512, 1024])
@pytest.mark.parametrize("at", [0, 77, 127])
def test_route_large_scores_beside_small_ones(E, at):
    """Softmax: the error of a score near 1 is far larger than that of one near 0, so a large one below both of the
    keys at the border may belong above them."""
    l = np.full((1, E), np.log(7e-8), np.float32)
    l[0, at] = 0.0
    p = np.exp(l[0].astype(np.float64))
    p /= p.sum()
    bias = np.full(E, -1.0, np.float32)
    bias[at] = -0.99
    top = p[at] + float(bias[at])
    for below in [(2e-7, 1.2e-6), (1e-7, 9e-7), (3e-7, 2e-6)]:
        b = bias.copy()
        others = [e for e in (5, 60, 100) if e != at][:2]
        for e, d in zip(others, below):
            b[e] = np.float32(top - d - p[e])
        check_route(l, b, 1, False)
        check_route(l, b, 2, False)
        check_route(l, b, 3, False)


def test_route_masks_in_the_bias():
    """Experts masked by a bias of -inf, up to leaving fewer than k; +inf forces a choice."""
    rng = np.random.default_rng(9)
    l = rng.standard_normal((40, 64)).astype(np.float32)
    for n in (60, 20, 8, 5, 0):
        bias = (0.05 * rng.standard_normal(64)).astype(np.float32)
        bias[rng.permutation(64)[:64 - n]] = -np.inf
        for sigmoid in (True, False):
            check_route(l, bias, 8, sigmoid)
    bias = np.zeros(64, np.float32)
    bias[[7, 50]] = np.inf
    check_route(l, bias, 4)


def test_route_groups_of_unequal_precision():
    """A group whose two keys are large and of opposite sign has a score of far larger error than its neighbours': it
    may belong above both groups at the border."""
    rng = np.random.default_rng(12)
    sig = lambda x: 1.0 / (1.0 + np.exp(-x.astype(np.float64)))
    rows, bias = [], np.array([1000.0, -1000.0, 0.0, 0.0, 0.0, 0.0], np.float32)
    while len(rows) < 40:
        x = rng.uniform(-1, 1, 2).astype(np.float32)
        true = sig(x).sum()
        f32 = float(np.float32(1000.0) + np.float32(sig(x)[0])) + float(np.float32(-1000.0) + np.float32(sig(x)[1]))
        if true - f32 < 4e-5:
            continue
        # the other two groups 2e-5 and 3e-5 below its true score, above its fp32 one
        want = np.array([true - 2e-5, true - 3e-5]) / 2
        y = np.log(want / (1 - want)).astype(np.float32)
        rows.append([x[0], x[1], y[0], y[0], y[1], y[1]])
    l = np.array(rows, np.float32)
    check_route(l, bias, 2, True, 3, 1)
    check_route(l, bias, 2, True, 3, 2)


def test_route_gates_of_scores_below_fp32():
    """Renormalised gates are ratios: they exist where the scores themselves are below fp32's range."""
    rng = np.random.default_rng(10)
    for base in (-80.0, -88.0, -95.0, -120.0, -700.0):
        l = (base + rng.uniform(-3, 3, (20, 64))).astype(np.float32)
        check_route(l, None, 8, True)
        check_route(l, None, 8, True, scale=2.5, n_group=4, topk_group=2, top2=False)
        check_route(l, None, 8, True, renorm=False)
        l[:, 5] = 30.0                                     # softmax: one that takes all, kept out by its bias
        bias = np.zeros(64, np.float32)
        bias[5] = -5.0
        check_route(l, bias, 8, False)
        check_route(l, None, 8, False)
    l = np.full((3, 64), -np.inf, np.float32)
    l[1, 40] = 1.0
    for sigmoid in (True, False):
        check_route(l, None, 8, sigmoid, renorm=False)


# ------------------------------------------------------------------ norm

@pytest.mark.parametrize("H", [256, 2304, 10240])
@pytest.mark.parametrize("T", [4, 700])
@pytest.mark.parametrize("off", [0, 1])
@pytest.mark.parametrize("fmt,g,top", [("Q8K", 256, 127.0), ("E4M3_G128", 128, 448.0), ("E4M3_ROW", 0, 448.0),
                                       ("INT8_ROW", 0, 127.0)])
def test_norm_zero_rows_without_eps(H, T, off, fmt, g, top):
    """eps = 0: rows of zeros, and rows whose squares are below fp32's range, have codes, scales and y of 0."""
    x, w = rnd((T, H), 3), 1 + 0.2 * rnd((H,), 4)
    x[1] = 0.0
    x[2] *= 1e-30
    xb = torch.zeros(T, H + off, device="cuda")
    xb[:, off:] = x.cuda()
    q = torch.full((T, H), 5.0, device="cuda").to(torch.float8_e4m3fn if top == 448.0 else torch.int8)
    d = torch.full((T, -(-H // (g or H))), 9.0, device="cuda")
    bs = torch.full((T, H // 16), 9, dtype=torch.int16, device="cuda") if fmt == "Q8K" else None
    y = torch.full((T, H), 9.0, device="cuda")
    moe.moe_add_rmsnorm(xb[:, off:], w.cuda(), 0.0, y=y, q_fmt=getattr(moe, "NORM_Q_" + fmt), q=q, d=d, bsum16=bs)
    for t in (1, 2):
        assert (y[t] == 0).all() and (q[t].float() == 0).all() and (d[t] == 0).all()
        assert bs is None or (bs[t] == 0).all()
    key = {"Q8K": "q8k", "E4M3_G128": "g128", "E4M3_ROW": "e4m3", "INT8_ROW": "int8"}[fmt]
    keep = [i for i in range(T) if i not in (1, 2)]
    check_norm(x[keep], None, w, 0.0, 0.0, None, y[keep], q[keep], d[keep], None if bs is None else bs[keep], key)


# ------------------------------------------------------------------ attention

@pytest.mark.parametrize("D", [64, 128, 256, 80])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 3])
def test_attention_largest_window(D, window):
    """A window as large as its type, with tokens that stand before the first key."""
    c = Cache([5, 40, 2], [2, 7, 50], 2, D, 16, BF16, 86)
    q, out, lse, ws = attend(c, 4, D, 0.1, window, BF16, 87)
    assert status(ws) == 0
    want, wl, tol, ltol = block_ref.attention(q, c.k, c.v, c.table, c.q_lens, c.kv_lens, 0.1, 0, BF16)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    none = torch.isneginf(wl)
    gl = lse.cpu().double()
    assert torch.equal(torch.isneginf(gl), none) and ((gl - wl).abs()[~none] <= ltol[~none]).all()


# the division of work in which most CTAs hold parts of two items
SHARED = ([1] * 100, [i * 131 % 4000 + 500 for i in range(100)], 8, 1)


@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("q_lens,kv_lens,hq,hkv", [SHARED, ([1, 1], [3000, 50], 16, 2)])
def test_attention_gives_up_waiting_for_parts(q_lens, kv_lens, hq, hkv, D):
    """Counters that never reach the number of parts: every CTA's wait runs out after a second, on the first of its
    items as on the second, the call ends with an error, and a zeroed workspace serves the next one."""
    c = Cache(q_lens, kv_lens, hkv, D, 64, BF16, 90)
    ws = torch.zeros(moe.moe_paged_attention_workspace_size(hq, hkv, D), dtype=torch.uint8, device="cuda")
    q, out, lse, _ = attend(c, hq, D, 0.1, 0, BF16, 91, ws=ws)
    good = out.clone()
    assert status(ws) == 0
    ws[16:16 + 4 * 160].view(torch.int32).fill_(2 ** 30)     # an increment takes these to 0, not on
    attend(c, hq, D, 0.1, 0, BF16, 91, ws=ws)
    assert status(ws) == moe.MOE_ERR_DEVICE_TIMEOUT
    ws.zero_()
    out = attend(c, hq, D, 0.1, 0, BF16, 91, ws=ws)[1]
    assert status(ws) == 0 and torch.equal(out.view(torch.int16), good.view(torch.int16))


@pytest.mark.parametrize("n,T,kv,hq", [(4, 40, 100, 4), (31, 300, 500, 16), (64, 40, 200, 4), (8192, 8192, 32768, 128),
                                       (8192, 8192, 49152, 128)])
@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_sequences_that_share_rows(n, T, kv, hq, D):
    """cu_q goes up and down, so that every other sequence names all rows: far more work than the call's sizes allow,
    up to more than 32 bits count.  Reported, and nothing is computed."""
    hkv, page = (8, 64) if hq == 128 else (2, 64)
    pages = -(-kv // page)
    kc = torch.zeros(pages, page, hkv, D, dtype=BF16, device="cuda")
    table = torch.arange(pages, dtype=torch.int32, device="cuda").repeat(n, 1)
    cu = torch.tensor([0 if b % 2 == 0 else T for b in range(n + 1)], dtype=torch.int32, device="cuda")
    lens = torch.full((n,), kv, dtype=torch.int32, device="cuda")
    q = torch.zeros(T, hq, D, dtype=BF16, device="cuda")
    out = torch.full((T, hq, D), 5.0, dtype=BF16, device="cuda")
    ws = torch.zeros(moe.moe_paged_attention_workspace_size(hq, hkv, D), dtype=torch.uint8, device="cuda")
    moe.moe_paged_attention(q, kc, kc, table, cu, lens, 0.1, out, ws)
    assert status(ws) == moe.MOE_ERR_DEVICE_BOUNDS
    assert (out == 5.0).all()
    cu = torch.tensor([0, T] + [T] * (n - 1), dtype=torch.int32, device="cuda")     # in order: the first has all rows
    moe.moe_paged_attention(q, kc, kc, table, cu, lens, 0.1, out, ws)
    assert status(ws) == 0 and (out == 0.0).all()


def positions(c):
    """Position of each token in its sequence, and the sequence."""
    pos, seq = [], []
    for b, (n, kv) in enumerate(zip(c.q_lens, c.kv_lens)):
        pos += list(range(kv - n, kv))
        seq += [b] * n
    return pos, seq


def check_special(c, hq, D, window, dtype, bad_v, bad_k=(), seed=81):
    """bad_v: (sequence, key, head, column, value) that are not finite, bad_k: (sequence, key, head) whose key is NaN.
    Rows that see none of them are as if they were 0; a row that sees a value has no finite number in its column; a
    row that sees a key has NaN everywhere."""
    page, hkv = c.k.shape[1], c.k.shape[2]
    G = hq // hkv
    clean_k, clean_v = c.k.clone(), c.v.clone()
    for b, j, h, col, v in bad_v:
        p = int(c.table[b, j // page])
        c.v[p, j % page, h, col] = v
        clean_v[p, j % page, h, col] = 0.0
    for b, j, h in bad_k:
        c.k[int(c.table[b, j // page]), j % page, h, D // 2] = NAN
    c.dk.copy_(c.k), c.dv.copy_(c.v)
    q, out, lse, ws = attend(c, hq, D, 0.1, window, dtype, seed)
    assert status(ws) == 0
    want, wl, tol, ltol = block_ref.attention(q, clean_k, clean_v, c.table, c.q_lens, c.kv_lens, 0.1, window, dtype)
    pos, seq = positions(c)
    got, gl = out.cpu().double(), lse.cpu().double()
    extra = torch.zeros_like(want)
    void = torch.zeros(c.T, hq, dtype=torch.bool)
    for t in range(c.T):
        sees = lambda b, j: seq[t] == b and j <= pos[t] and (not window or j > pos[t] - window)
        for b, j, h, col, v in bad_v:
            if sees(b, j):
                extra[t, h * G:(h + 1) * G, col] += v
        for b, j, h in bad_k:
            if sees(b, j):
                void[t, h * G:(h + 1) * G] = True
    fine = torch.isfinite(extra) & ~void.unsqueeze(2)
    assert (extra[fine] == 0).all()
    assert torch.isnan(got[void]).all() and torch.isnan(gl[void]).all()
    assert ((got - want).abs() <= tol)[fine].all()
    none = torch.isneginf(wl) & ~void
    assert torch.isneginf(gl[none]).all()
    rest = ~none & ~void
    assert ((gl - wl).abs()[rest] <= ltol[rest]).all()
    # (not finite, not which: the weight of a far key may be 0 in 16 bits, and 0 times infinity is NaN)
    assert not torch.isfinite(got[~torch.isfinite(extra) & ~void.unsqueeze(2)]).any()
    return ws


@pytest.mark.parametrize("D", [64, 128, 256, 80])
@pytest.mark.parametrize("dtype", [BF16, F16])
@pytest.mark.parametrize("q_lens,kv_lens", [([1, 2], [40, 33]), ([1], [6000]), ([150, 3], [200, 60])])
def test_attention_of_keys_and_values_that_are_not_finite(q_lens, kv_lens, D, dtype):
    """What every row sees: NaN keys make rows NaN in out and in lse, values that are not finite reach their column."""
    c = Cache(q_lens, kv_lens, 2, D, 32, dtype, 80)
    check_special(c, 6, D, 0, dtype, [(0, 3, 0, 5, INF), (0, 20, 1, 7, -INF), (0, 2, 1, D - 1, NAN)])
    c = Cache(q_lens, kv_lens, 2, D, 32, dtype, 82)
    check_special(c, 6, D, 0, dtype, [], [(0, 7, 1)])


@pytest.mark.parametrize("D", [64, 128, 256, 80])
@pytest.mark.parametrize("q_lens,kv_lens,hq,window", [
    ([4, 5], [40, 33], 4, 0), ([4], [4000], 16, 0), ([150, 3], [200, 60], 6, 0), ([300], [300], 2, 0),
    ([4, 9], [70, 300], 8, 20), ([150], [600], 4, 33), ([150], [500], 4, 1), ([40], [3000], 32, 1000), ([1], [500], 8, 37)])
def test_attention_hidden_values_do_not_matter(q_lens, kv_lens, hq, window, D):
    """Values that are not finite, at keys that a row does not see: of later tokens, and before the window, next to what
    it sees.  The rows that do see them have them."""
    page = 32
    c = Cache(q_lens, kv_lens, 2, D, page, F16, 84)
    bad, keys = [], []
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        new = range(kv - n, kv)
        for i, j in enumerate(new):                        # most of the later tokens; the first stays clean
            if i and (n < 20 or i % 7 == 1):
                bad.append((b, j, i % 2, (11 * i) % D, [INF, -INF, NAN][i % 3]))
        if n > 1:
            bad += [(b, kv - 1, 1, 2, -INF), (b, kv - 1, 0, 2, INF)]
            keys.append((b, kv - 1, 0))
        if window:
            low = kv - n + 1 - window                      # the first key that the first token sees
            for j in range(max(0, low - page), max(0, low)):
                bad.append((b, j, j % 2, (5 * j) % D, NAN))
            for i in range(1, n, 5):                       # seen by the first tokens, not by the later ones
                if 0 <= low + i - 1 < kv - n:
                    bad.append((b, low + i - 1, i % 2, (3 * i + 1) % D, INF))
    check_special(c, hq, D, window, F16, bad)
    c = Cache(q_lens, kv_lens, 2, D, page, F16, 85)
    check_special(c, hq, D, window, F16, bad[:3], keys)


@pytest.mark.parametrize("D", [64, 128, 256])
def test_attention_many_small_weights_in_fp16(D):
    """One key far above many others in the same run of tiles: each of those has a weight near 2^-20 of the largest, all
    of them together a good part of the sum.  Half a step's relative error asks for weights that are normal numbers.
    (Three hundred sequences share the keys, so that every one is whole.)"""
    kv, page, n = 16384, 64, 300
    k, v = torch.zeros(kv // page, page, 1, D, dtype=F16), torch.ones(kv // page, page, 1, D, dtype=F16)
    k[0, 0], v[0, 0] = 1.0, 0.0
    table = torch.arange(kv // page, dtype=torch.int32).view(1, -1)
    cu = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    lens = torch.full((n,), kv, dtype=torch.int32, device="cuda")
    q = torch.ones(n, 1, D, dtype=F16)
    out = torch.empty(n, 1, D, dtype=F16, device="cuda")
    lse = torch.empty(n, 1, device="cuda")
    ws = torch.zeros(moe.moe_paged_attention_workspace_size(1, 1, D), dtype=torch.uint8, device="cuda")
    scale = float(np.log(2.0 ** 24 / 10.45)) / D          # weights of 10.45 * 2^-24
    moe.moe_paged_attention(q.cuda(), k.cuda(), v.cuda(), table.cuda().repeat(n, 1), cu, lens, scale, out, ws, lse=lse)
    assert status(ws) == 0
    want, wl, tol, ltol = block_ref.attention(q[:1], k, v, table, [1], [kv], scale, 0, F16)
    assert ((out.cpu().double() - want).abs() <= tol).all()
    assert ((lse.cpu().double() - wl).abs() <= ltol).all()
