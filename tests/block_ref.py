"""Plain 64-bit implementations of the decoder-block operators, and bounds on what fp32 arithmetic and one
rounding to a narrower type may change.  numpy / torch on the CPU only."""
import numpy as np
import torch

U32 = 2.0 ** -24                                              # half a step of fp32, relative
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}
TINY = {torch.float32: 2.0 ** -149, torch.bfloat16: 2.0 ** -133, torch.float16: 2.0 ** -25}   # half a subnormal step or more


def norm(x, residual, w, eps, offset=0.0):
    """(s, z) in fp64."""
    s = x.double() if residual is None else x.double() + residual.double()
    return s, s / torch.sqrt((s * s).mean(1, keepdim=True) + eps) * (w.double() + offset)


def route(logits, bias, k, sigmoid, n_group, topk_group, top2, renorm, scale):
    """ids [T, k], gates [T, k] by the definition, one token at a time."""
    T, E = logits.shape
    gs = E // n_group
    ids, gates = np.zeros((T, k), np.int32), np.zeros((T, k))
    for t in range(T):
        l = np.where(np.isnan(logits[t]), -np.inf, logits[t].astype(np.float64))
        if sigmoid:
            with np.errstate(over="ignore"):
                p = 1.0 / (1.0 + np.exp(-l))
        elif l.max() == -np.inf:
            p = np.zeros(E)
        else:
            with np.errstate(invalid="ignore"):
                e = np.where(l == l.max(), 1.0, np.exp(l - l.max()))
            p = e / e.sum()
        key = p if bias is None else p + bias.astype(np.float64)
        order = l if bias is None else key
        live = np.ones(E, bool)
        if n_group > 1:
            score = []
            for g in range(n_group):
                part = np.sort((key if top2 or bias is not None else l)[g * gs:(g + 1) * gs])[::-1]
                score.append(part[0] + part[1] if top2 and gs > 1 else part[0])
            best = sorted(range(n_group), key=lambda g: (-score[g], g))[:topk_group]
            live = np.isin(np.arange(E) // gs, best)
        pick = sorted(np.nonzero(live)[0], key=lambda e: (-order[e], e))[:k]
        ids[t] = pick
        g = p[pick]
        if renorm:
            g = g / g.sum() if g.sum() > 0 else np.zeros(k)
        gates[t] = g * scale
    return ids, gates


def attention(q, k_cache, v_cache, table, q_lens, kv_lens, scale, window, dtype):
    """out, lse and their bounds, in fp64.  q [T, Hq, D]; caches [pages, page, Hkv, D]."""
    T, Hq, D = q.shape
    page, hkv = k_cache.shape[1:3]
    G = Hq // hkv
    out, lse = torch.zeros(T, Hq, D, dtype=torch.float64), torch.full((T, Hq), -np.inf, dtype=torch.float64)
    out_tol, lse_tol = torch.zeros(T, Hq, D, dtype=torch.float64), torch.zeros(T, Hq, dtype=torch.float64)
    u = HALF_STEP[dtype]
    at = 0
    for b, (n, kv) in enumerate(zip(q_lens, kv_lens)):
        if n and kv:
            ids = table[b, :-(-kv // page)].long()
            keys = k_cache[ids].reshape(-1, hkv, D)[:kv].double()
            vals = v_cache[ids].reshape(-1, hkv, D)[:kv].double()
            pos = torch.arange(kv - n, kv)[:, None]
            j = torch.arange(kv)[None]
            hidden = (j > pos) | ((j <= pos - window) if window else torch.zeros(1, 1, dtype=torch.bool))
            for h in range(Hq):
                qq, kk, vv = q[at:at + n, h].double(), keys[:, h // G], vals[:, h // G]
                a = (qq @ kk.T * scale).masked_fill(hidden, -np.inf)
                big = (qq.abs() @ kk.abs().T * abs(scale)).masked_fill(hidden, 0.0).amax(1)
                m = a.amax(1, keepdim=True).clamp(min=-1e300)
                p = torch.exp(a - m)
                l = p.sum(1, keepdim=True)
                w = torch.where(l > 0, p / l, torch.zeros_like(p))
                out[at:at + n, h] = w @ vv
                lse[at:at + n, h] = (m + torch.log(l)).squeeze(1)
                # a score: a dot product of D products, scaled and shifted (the shift by the running maximum
                # rounds at its size); a weight: exp2 within 2 ulp, sums of at most kv terms in any order
                ds = ((D + 8) * U32 * big)[:, None]
                rel = 2 * ds + (16 + 8 + kv / 64) * U32
                A = w @ vv.abs()
                out_tol[at:at + n, h] = 1.01 * (A * (u + 2 * rel) + out[at:at + n, h].abs() * u) + TINY[dtype]
                lse_tol[at:at + n, h] = (rel + 4 * U32 * (lse[at:at + n, h].abs()[:, None] + 1)).squeeze(1).nan_to_num(0.0, posinf=0.0)
        at += n
    return out, lse, out_tol, lse_tol
