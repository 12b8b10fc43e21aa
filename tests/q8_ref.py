"""Plain forms of the 8-bit cache's operators on the CPU, and a cache to test them with."""
import numpy as np
import torch

import block_quantized_routed_gb300 as moe

E4M3, INT8 = torch.float8_e4m3fn, torch.int8
TOP = {E4M3: 448.0, INT8: 127.0}


def quantise(x, fmt):
    """Codes and scales of the vectors in the last dimension, by the definition, in IEEE fp32."""
    x = x.float().numpy()
    peak = np.abs(x).max(-1)
    x = np.where(peak[..., None] == 0, np.float32(0), x)   # zeros of either sign have code 0
    bad = ~np.isfinite(peak) | np.isnan(x).any(-1)
    d = np.where(peak > 0, np.maximum(peak / np.float32(TOP[fmt]), np.float32(2.0 ** -126)), np.float32(0)).astype(np.float32)
    d = np.where(bad, np.float32(1), d)
    z = np.where(bad[..., None], np.float32(0), x) / np.where(d > 0, d, np.float32(1))[..., None]
    assert z.dtype == np.float32
    if fmt == E4M3:
        codes = torch.from_numpy(np.clip(z, -448, 448)).to(E4M3)
    else:
        z = z.astype(np.float64)   # halves away from zero: exact in 64 bits
        codes = torch.from_numpy(np.clip(np.trunc(z + np.copysign(0.5, z)), -127, 127).astype(np.int8))
    return codes, torch.from_numpy(np.where(bad, np.float32(np.nan), d))


def code_values(codes):
    """The numbers that codes stand for, in fp64."""
    if codes.dtype == INT8:
        return codes.double()
    b = codes.view(torch.uint8).int()
    e, m = (b >> 3) & 15, (b & 7).double()
    mag = torch.where(e > 0, (1 + m / 8) * torch.pow(2.0, e.double() - 7), m / 8 * 2.0 ** -6)
    mag = torch.where((b & 127) == 127, torch.full_like(mag, float("nan")), mag)
    return torch.where(b >= 128, -mag, mag)


class Q8Cache:
    """Sequences of given lengths in a shuffled paged cache of random codes, on the GPU; the CPU's copy beside it.
    layout: rows ([pages, page, Hkv, D]), heads ([pages, Hkv, page, D]) or odd (rows with a gap, off 16 bytes)."""

    def __init__(self, lens, Hkv, D, page, fmt, seed=0, layout="rows", spare=2):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // page) for n in lens]
        pages, most = sum(need) + spare, max(1, max(need, default=1))
        order = torch.randperm(pages, generator=g).int()
        self.table = torch.zeros(len(lens), most, dtype=torch.int32)
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.lens, self.page, self.fmt, self.pages, self.Hkv, self.D = lens, page, fmt, pages, Hkv, D
        codes, scales = [], []
        for _ in range(2):
            x = torch.randn(pages, page, Hkv, D, generator=g) * (1 + 5 * (torch.rand(Hkv, D, generator=g) < 0.05))
            c, d = quantise(x * torch.exp(torch.randn(pages, page, Hkv, 1, generator=g)), fmt)
            codes.append(c)
            scales.append(d)
        self.kc, self.vc, self.ks, self.vs = *codes, *scales

        def place(t):
            raw = t.view(torch.uint8).cuda() if t.dtype == E4M3 else t.cuda()
            if layout == "heads":
                out = raw.transpose(1, 2).contiguous().transpose(1, 2)
            elif layout == "odd" and t.dim() == 4:
                out = torch.empty(pages, page, Hkv, D + 3, dtype=raw.dtype, device="cuda")[..., 1:D + 1]
                out.copy_(raw)
            else:
                out = raw
            return out.view(E4M3) if t.dtype == E4M3 else out
        self.gkc, self.gvc, self.gks, self.gvs = (place(t) for t in (self.kc, self.vc, self.ks, self.vs))
        self.gtable = self.table.cuda()
        self.kv_len = torch.tensor(lens, dtype=torch.int32, device="cuda")

    def sequence(self, b, name):
        """fp64 values [kv, Hkv, D] of a sequence."""
        n = self.lens[b]
        ids = self.table[b, :-(-n // self.page)].long()
        c, d = (self.kc, self.ks) if name == "k" else (self.vc, self.vs)
        return (code_values(c.view(torch.uint8)[ids].view(c.dtype)) * d[ids].double().unsqueeze(-1)).reshape(-1, self.Hkv, self.D)[:n]


def status(ws):
    return moe.moe_get_status(ws)


def new_ws(n=16):
    return torch.zeros(n, dtype=torch.uint8, device="cuda")


U32 = 2.0 ** -24                                              # half a step of fp32, relative
HALF_STEP = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}


def attention(q, c, q_lens, scale, window):
    """out, lse and their bounds in fp64 for q [T, Hq, D] over the cache c."""
    T, Hq, D = q.shape
    G = Hq // c.Hkv
    inf = float("inf")
    out, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((T, Hq), -inf, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    at = 0
    for b, n in enumerate(q_lens):
        kv = c.lens[b]
        if n and kv:
            keys, vals = c.sequence(b, "k"), c.sequence(b, "v")
            ids = c.table[b, :-(-kv // c.page)].long()
            e = c.vs[ids].double().reshape(-1, c.Hkv)[:kv]
            pos = torch.arange(kv - n, kv)[:, None]
            j = torch.arange(kv)[None]
            hidden = (j > pos) | ((j <= pos - window) if window else torch.zeros(1, 1, dtype=torch.bool))
            for h in range(Hq):
                qq, kk, vv = q[at:at + n, h].double(), keys[:, h // G], vals[:, h // G]
                a = (qq @ kk.T * scale).masked_fill(hidden, -inf)
                big = (qq.abs() @ kk.abs().T * abs(scale)).masked_fill(hidden, 0.0).amax(1)
                small = (qq.abs().amax(1, keepdim=True) @ kk.abs().sum(1)[None] * abs(scale)).masked_fill(hidden, 0.0).amax(1)
                m = a.amax(1, keepdim=True).clamp(min=-1e300)
                p = torch.exp(a - m)
                l = p.sum(1, keepdim=True)
                w = torch.where(l > 0, p / l, torch.zeros_like(p))
                out[at:at + n, h] = w @ vv
                lse[at:at + n, h] = (m + torch.log(l)).squeeze(1)
                # a score: a dot product of D products, the query in fp16 relative to its largest element (what is
                # subnormal there is off by 2^-38 of it), scaled twice and shifted; a weight: exp2 within 2 ulp, the
                # logarithm of its scale within 2^-22, one rounding to fp16, below fp16's normal numbers off by 2^-33
                # of the largest; sums of at most kv terms in any order
                ds = ((D + 10) * U32 * big + 2.0 ** -38 * small)[:, None]
                rel = 2 * ds + (16 + 16 + kv / 64) * U32
                weighted = w * e[:, h // G]
                floor = kv * 2.0 ** -33 * 480 * torch.nan_to_num(weighted).amax(1, keepdim=True)
                A = w @ vv.abs()
                u = HALF_STEP[q.dtype]
                out_tol[at:at + n, h] = 1.01 * (A * (2.0 ** -11 + 2 * rel) + out[at:at + n, h].abs() * u + floor) + TINY[q.dtype]
                lse_tol[at:at + n, h] = (rel + 4 * U32 * (lse[at:at + n, h].abs()[:, None] + 1)).squeeze(1).nan_to_num(0.0, posinf=0.0)
        at += n
    return out, lse, out_tol, lse_tol
