"""Cases, plain forms and 64-bit definitions of the operators of a decoder block with an 8-bit key/value cache.

  append  a chunk's new keys and values quantised as they are written into the pages of a cache
          (moe_kv_append_q8): e4m3 or int8 codes, one fp32 scale per token and head
  read    the cache's sequences read back as 16- or 32-bit rows (moe_kv_read_q8)
  attn    attention of single tokens and verify windows over that cache, which is read as it lies
          (moe_paged_attention_q8)
  linear  the block's dense projections: a matrix product with bias, activation and residual in its epilogue
          (moe_linear)

`own` chooses between the plain form (elementary torch operations in 32 bits) and the package's public calls.
Both take what prepare() gives.
"""
import math
import random

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn,
          "int8": torch.int8}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "": 0}
TOP = {"e4m3": 448.0, "int8": 127.0}
LEAST = 2.0 ** -126     # the smallest scale of a vector that is not all zeros


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one new token of each of 64 requests: latency
        {"name": "append_decode", "op": "append", "B": 64, "q": 1, "kv": 2048, "hkv": 4, "D": 128, "page": 64,
         "x": "bf16", "fmt": "e4m3", "ragged": False, "lens": 1},
        # prompt chunks of three requests, pages that end inside a chunk
        {"name": "append_chunk", "op": "append", "B": 3, "q": 4096, "kv": 8192, "hkv": 8, "D": 128, "page": 32,
         "x": "bf16", "fmt": "e4m3", "ragged": True, "lens": 2},
        # a few conversations brought back to 16 bits, int8 codes, narrow heads
        {"name": "read_ragged", "op": "read", "B": 7, "kv": 1999, "hkv": 8, "D": 64, "page": 16, "x": "f16",
         "fmt": "int8", "lens": 3},
        # long pasts read back before a prompt chunk's attention on the tensor cores
        {"name": "read_long", "op": "read", "B": 3, "kv": 32768, "hkv": 8, "D": 128, "page": 64, "x": "bf16",
         "fmt": "e4m3", "lens": 4},
        # the next token of one short conversation: latency
        {"name": "attn_token", "op": "attn", "B": 1, "q": 1, "kv": 777, "hq": 16, "hkv": 2, "D": 256, "page": 16,
         "window": 0, "x": "bf16", "fmt": "e4m3", "ragged": False, "lens": 5},
        # the next tokens of 48 conversations of different lengths: the cache is read once
        {"name": "attn_decode", "op": "attn", "B": 48, "q": 1, "kv": 8192, "hq": 32, "hkv": 4, "D": 128, "page": 64,
         "window": 0, "x": "bf16", "fmt": "e4m3", "ragged": True, "lens": 6},
        # verify windows of up to 4 drafts with a sliding window, heads shared by fives, int8 codes
        {"name": "attn_verify", "op": "attn", "B": 16, "q": 4, "kv": 4001, "hq": 40, "hkv": 8, "D": 64, "page": 32,
         "window": 1024, "x": "f16", "fmt": "int8", "ragged": True, "lens": 7},
        # four very long contexts: memory bound
        {"name": "attn_long", "op": "attn", "B": 4, "q": 1, "kv": 131072, "hq": 64, "hkv": 8, "D": 128, "page": 64,
         "window": 0, "x": "bf16", "fmt": "e4m3", "ragged": True, "lens": 8},
        # queries, keys and values of one decoded token of a 2048-wide model: the weights are read once
        {"name": "linear_token", "op": "linear", "T": 1, "K": 2048, "N": 5120, "x": "bf16", "bias": True, "act": "none",
         "res": "", "out": "bf16"},
        # attention outputs of drafts projected onto the fp32 residual stream
        {"name": "linear_drafts", "op": "linear", "T": 37, "K": 4096, "N": 6144, "x": "bf16", "bias": False,
         "act": "none", "res": "f32", "out": "f32"},
        # ragged prompts through a dense layer of an odd width
        {"name": "linear_ragged", "op": "linear", "T": 1021, "K": 2048, "N": 7001, "x": "f16", "bias": True,
         "act": "gelu", "res": "", "out": "f16"},
        # a prompt chunk: compute bound
        {"name": "linear_chunk", "op": "linear", "T": 8192, "K": 4096, "N": 5120, "x": "bf16", "bias": True,
         "act": "silu", "res": "bf16", "out": "bf16"},
    ]


def _log(rng, lo, hi):
    """An integer of [lo, hi], spread over its logarithm."""
    return max(lo, min(hi, int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))))


def draw(rng):
    op = rng.choice(["append", "read", "attn", "attn", "linear", "linear"])
    x = rng.choice(["bf16", "f16"])
    if op == "linear":
        c = {"op": op, "T": _log(rng, 1, 8192), "K": 8 * _log(rng, 8, 1024), "N": _log(rng, 64, 8192), "x": x,
             "bias": rng.random() < 0.6, "act": rng.choice(["none", "none", "relu", "silu", "gelu", "gelu_tanh"]),
             "res": rng.choice(["", x, "f32"]), "out": rng.choice([x, "f32"])}
        while c["T"] * c["K"] * c["N"] > 8192 * 4096 * 5120:
            c["T"] //= 2
        return c
    D = rng.choice([64, 128, 256])
    c = {"op": op, "hkv": rng.choice([1, 2, 4, 8]), "D": D, "page": rng.choice([16, 32, 48, 64, 128, 256]), "x": x,
         "fmt": rng.choice(["e4m3", "int8"]), "lens": rng.randrange(1 << 20)}
    if op == "read":
        c["x"] = rng.choice(["bf16", "f16", "f32"])
        c["B"], c["kv"] = _log(rng, 1, 32), _log(rng, 1, 32768)
        while c["B"] * c["kv"] * c["hkv"] * D > 1 << 25:
            c["kv"] //= 2
        return c
    c["ragged"] = True
    kind = rng.choice(["decode", "verify", "chunk"] if op == "append" else ["decode", "verify"])
    c["B"] = _log(rng, 1, 64) if kind != "chunk" else _log(rng, 1, 4)
    c["q"] = 1 if kind == "decode" else rng.randint(2, 16) if kind == "verify" else _log(rng, 17, 4096)
    if op == "attn":
        c["kv"] = max(c["q"], _log(rng, 1, 131072))
        c["hq"] = c["hkv"] * rng.choice([1, 2, 3, 4, 5, 6, 8, 16])
        c["window"] = rng.choice([0, 0, 0, _log(rng, 1, 4096)])
        most = 1 << 28
    else:
        c["kv"] = max(c["q"], _log(rng, 1, 8192))
        most = 1 << 22 if c["fmt"] == "int8" else 1 << 25
    while c["B"] * c["kv"] * c["hkv"] * D > most or op == "attn" and c["B"] * c["hq"] * c["q"] * c["kv"] > 1 << 26:
        c["kv"] = max(1, c["kv"] // 2)
        c["q"] = min(c["q"], c["kv"])
    return c


def lengths(c):
    """(new tokens, keys including them) of each sequence of a case; the first length is the longest."""
    rng = random.Random(c["lens"])
    q = c.get("q", 0)
    out = [(q, c["kv"])]
    for _ in range(c["B"] - 1):
        if c["op"] == "read":
            out.append((0, rng.randint(0, c["kv"])))
        else:
            n = rng.randint(1, q) if c["ragged"] else q
            out.append((n, rng.randint(n, max(n, c["kv"])) if c["ragged"] else rng.randint(c["kv"] // 2, c["kv"])))
    rng.shuffle(out)
    return out


def rows_of(c):
    """First row of each sequence in the rows that are read back, and their number: whole pages each."""
    at, first = 0, []
    for _, kv in lengths(c):
        first.append(at)
        at += -(-kv // c["page"]) * c["page"]
    return first, at


# ------------------------------------------------------------------ inputs

def _gen(seed, salt):
    return torch.Generator(device="cuda").manual_seed(seed * 1000003 + salt)


def _randn(shape, g, dtype=torch.float32):
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _quantise(x, fmt):
    """Codes and scales of vectors in the last dimension: d = max|x| / top, code = x / d rounded (int8: halves away
    from zero), a vector of zeros has d = 0."""
    x = x.float()
    peak = x.abs().amax(-1)
    d = torch.where(peak > 0, (peak / TOP[fmt]).clamp_min(LEAST), torch.zeros_like(peak))
    z = x / torch.where(d > 0, d, torch.ones_like(d)).unsqueeze(-1)
    if fmt == "e4m3":
        return z.clamp(-448.0, 448.0).to(torch.float8_e4m3fn), d
    return (torch.sign(z) * torch.floor(z.abs() + 0.5)).clamp(-127.0, 127.0).to(torch.int8), d


def _values(codes, d, dtype):
    return (codes.float() * d.unsqueeze(-1)).to(dtype)


def prepare(case, seed):
    c = dict(case)
    return _prepare_linear(c, seed) if c["op"] == "linear" else _prepare_cache(c, seed)


def _prepare_linear(c, seed):
    g, dt = _gen(seed, 1), DTYPES[c["x"]]
    T, K, N = c["T"], c["K"], c["N"]
    s = {"c": c, "x": _randn((T, K), g, dt), "w": (_randn((N, K), g) * K ** -0.5).to(dt)}
    s["bias"] = 0.5 * _randn((N,), g) if c["bias"] else None
    s["res"] = (2.0 * _randn((T, N), g)).to(DTYPES[c["res"]]) if c["res"] else None
    s["out"] = torch.empty((T, N), dtype=DTYPES[c["out"]], device="cuda")
    return s


def _prepare_cache(c, seed):
    g, dt = _gen(seed, 2), DTYPES[c["x"]]
    lens = lengths(c)
    page, hkv, D, fmt = c["page"], c["hkv"], c["D"], c["fmt"]
    need = [-(-kv // page) for _, kv in lens]
    pages, most = sum(need) + 3, max(1, max(need))
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    table = torch.zeros((len(lens), most), dtype=torch.int32, device="cuda")
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    cu = torch.zeros(len(lens) + 1, dtype=torch.int32)
    cu[1:] = torch.cumsum(torch.tensor([n for n, _ in lens], dtype=torch.int32), 0)
    T = int(cu[-1])
    s = {"c": c, "lens": lens, "table": table, "cu": cu.cuda(),
         "kv_len": torch.tensor([kv for _, kv in lens], dtype=torch.int32, device="cuda")}
    loud = 1.0 + 6.0 * (torch.rand((hkv, D), generator=g, device="cuda") < 0.03).float()  # keys have loud channels
    mean = 0.3 * _randn((hkv, D), g)
    for name in ("k", "v"):
        codes = torch.empty((pages, page, hkv, D), dtype=DTYPES[fmt], device="cuda")
        scales = torch.empty((pages, hkv, page), device="cuda").transpose(1, 2)  # a head's scales lie together
        step = max(1, (1 << 25) // (page * hkv * D))
        for i in range(0, pages, step):
            x = _randn((min(step, pages - i), page, hkv, D), g)
            x = x * loud if name == "k" else x + mean
            codes[i:i + step], scales[i:i + step] = _quantise(x, fmt)
        s[name + "c"], s[name + "s"] = codes, scales
    if c["op"] == "read":
        first, rows = rows_of(c)
        s["first"] = torch.tensor(first, dtype=torch.int32, device="cuda")
        s["ko"] = torch.zeros((rows, hkv, D), dtype=dt, device="cuda")
        s["vo"] = torch.zeros((rows, hkv, D), dtype=dt, device="cuda")
    else:
        hq = c.get("hq", hkv)
        qkv = _randn((T, (hq + 2 * hkv) * D), g, dt).view(T, hq + 2 * hkv, D)  # one projection's output: strided views
        s["qn"], s["kn"], s["vn"] = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
        if c["op"] == "append":
            s["kn"].mul_(loud.to(dt))
    if c["op"] == "attn":
        s["scale"] = 0.7 / math.sqrt(D)
        s["out"] = torch.empty((T, hq, D), dtype=dt, device="cuda")
        s["lse"] = torch.empty((T, hq), device="cuda")
    if c["op"] == "append" and fmt == "int8":  # where the codes are turned into values
        s["kval"] = torch.empty(s["kc"].shape, dtype=torch.bfloat16, device="cuda")
        s["vval"] = torch.empty(s["vc"].shape, dtype=torch.bfloat16, device="cuda")
    if own:
        import block_quantized_routed_gb300 as moe
        n = moe.moe_paged_attention_q8_workspace_size(hq, hkv, D) if c["op"] == "attn" else 16
        s["ws"] = torch.zeros(n, dtype=torch.uint8, device="cuda")
    return s


# ------------------------------------------------------------------ the passes

def run(s):
    return {"append": _run_append, "read": _run_read, "attn": _run_attn, "linear": _run_linear}[s["c"]["op"]](s)


def _places(s):
    """Of each new token: its sequence, its number in the chunk and its position in the sequence."""
    cu = s["cu"].long()
    tok = torch.arange(s["kn"].shape[0], device="cuda")
    seq = torch.searchsorted(cu[1:].contiguous(), tok, right=True)
    i = tok - cu[seq]
    return seq, i, s["kv_len"].long()[seq] - (cu[seq + 1] - cu[seq]) + i


def _run_append(s):
    if own:
        import block_quantized_routed_gb300 as moe
        moe.moe_kv_append_q8(s["kn"], s["vn"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["kv_len"],
                             s["ws"])
    else:
        page = s["c"]["page"]
        seq, _, pos = _places(s)
        at, slot = s["table"].long()[seq, pos // page], pos % page
        for name in ("k", "v"):
            codes, d = _quantise(s[name + "n"], s["c"]["fmt"])
            s[name + "c"].view(torch.uint8)[at, slot] = codes.view(torch.uint8)
            s[name + "s"][at, slot] = d
    r = {"ks": s["ks"], "vs": s["vs"]}
    for name in ("k", "v"):
        if s["c"]["fmt"] == "int8":
            torch.mul(s[name + "c"], s[name + "s"].unsqueeze(-1), out=s[name + "val"])
            r[name] = s[name + "val"]
        else:
            r[name] = s[name + "c"]
    return r


def _run_read(s):
    if own:
        import block_quantized_routed_gb300 as moe
        moe.moe_kv_read_q8(s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["kv_len"], s["first"], s["ko"], s["vo"],
                           s["ws"])
        return {"k": s["ko"], "v": s["vo"]}
    page, kv_len, first = s["c"]["page"], s["kv_len"].long(), s["first"].long()
    row = torch.arange(s["ko"].shape[0], device="cuda")
    ends = torch.cumsum((kv_len + page - 1) // page * page, 0)      # each sequence has whole pages of rows
    seq = torch.searchsorted(ends, row, right=True)
    j = row - first[seq]
    row, seq, j = (t[j < kv_len[seq]] for t in (row, seq, j))
    at, slot = s["table"].long()[seq, j // page], j % page
    for name in ("k", "v"):
        s[name + "o"][row] = _values(s[name + "c"].view(torch.uint8)[at, slot].view(s[name + "c"].dtype),
                                     s[name + "s"][at, slot], s[name + "o"].dtype)
    return {"k": s["ko"], "v": s["vo"]}


def _run_attn(s):
    c = s["c"]
    if own:
        import block_quantized_routed_gb300 as moe
        moe.moe_paged_attention_q8(s["qn"], s["kc"], s["vc"], s["ks"], s["vs"], s["table"], s["cu"], s["kv_len"],
                                   s["scale"], s["out"], s["ws"], lse=s["lse"], window=c["window"])
        return {"out": s["out"], "lse": s["lse"]}
    hq, hkv, D, page = c["hq"], c["hkv"], c["D"], c["page"]
    G, B = hq // hkv, len(s["lens"])
    most_q, most_kv = max(n for n, _ in s["lens"]), max(kv for _, kv in s["lens"])
    seq, i, _ = _places(s)
    q = torch.zeros((B, most_q, hq, D), device="cuda")
    q[seq, i] = s["qn"].float()
    q = q.view(B, most_q, hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, hkv, G * most_q, D)
    j = torch.arange(most_kv, device="cuda")
    at = s["table"].long()[:, j // page]
    dt = s["kc"].dtype
    k = _values(s["kc"].view(torch.uint8)[at, j % page].view(dt), s["ks"][at, j % page], torch.float32)
    k = k.permute(0, 2, 3, 1)
    kv_len = s["kv_len"].long()
    last = (kv_len - (s["cu"][1:] - s["cu"][:-1]).long()).unsqueeze(1) + torch.arange(most_q, device="cuda")
    seen = j <= last.unsqueeze(2)
    if c["window"]:
        seen &= j > last.unsqueeze(2) - c["window"]
    seen &= (j < kv_len.unsqueeze(1)).unsqueeze(1)
    a = torch.matmul(q, k).mul_(s["scale"]).view(B, hkv, G, most_q, most_kv)
    del k
    a = a.masked_fill_(~seen[:, None, None], -math.inf)
    m = a.amax(4, keepdim=True).clamp_(min=-3e38)
    a = a.sub_(m).exp_()
    l = a.sum(4, keepdim=True)
    v = _values(s["vc"].view(torch.uint8)[at, j % page].view(dt), s["vs"][at, j % page], torch.float32)
    o = torch.matmul(a.view(B, hkv, G * most_q, most_kv), v.permute(0, 2, 1, 3)).view(B, hkv, G, most_q, D)
    o = torch.where(l > 0, o / l, torch.zeros_like(o)).permute(0, 3, 1, 2, 4).reshape(B, most_q, hq, D)
    lse = (m + torch.log(l)).squeeze(4).permute(0, 3, 1, 2).reshape(B, most_q, hq)
    return {"out": o[seq, i].to(s["out"].dtype), "lse": lse[seq, i]}


def _run_linear(s):
    c = s["c"]
    if own:
        import block_quantized_routed_gb300 as moe
        act = {"none": moe.ACT_NONE, "relu": moe.ACT_RELU, "silu": moe.ACT_SILU, "gelu": moe.ACT_GELU,
               "gelu_tanh": moe.ACT_GELU_TANH}[c["act"]]
        moe.moe_linear(s["x"], s["w"], s["out"], bias=s["bias"], act=act, residual=s["res"])
        return {"out": s["out"]}
    y = torch.matmul(s["x"].float(), s["w"].float().t())
    if s["bias"] is not None:
        y = y + s["bias"]
    if c["act"] == "relu":
        y = y.clamp_min(0.0)
    elif c["act"] == "silu":
        y = y / (1.0 + torch.exp(-y))
    elif c["act"] == "gelu":
        y = 0.5 * y * (1.0 + torch.erf(y * math.sqrt(0.5)))
    elif c["act"] == "gelu_tanh":
        y = 0.5 * y * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (y + 0.044715 * y * y * y)))
    if s["res"] is not None:
        y = y + s["res"].float()
    return {"out": y.to(s["out"].dtype)}


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c = case
    if c["op"] == "linear":
        T, K, N = c["T"], c["K"], c["N"]
        b = 2 * (T * K + N * K) + T * N * (BYTES[c["res"]] + BYTES[c["out"]]) + (4 * N if c["bias"] else 0)
        return {"bytes": b, "flops": 2 * T * K * N}
    lens = lengths(c)
    T, code = sum(n for n, _ in lens), c["hkv"] * (c["D"] + 4)  # a key's codes and scales
    if c["op"] == "append":
        return {"bytes": 2 * T * (code + c["hkv"] * c["D"] * 2) + 4 * sum(-(-n // c["page"]) for n, _ in lens),
                "flops": 0}
    keys, entries = sum(kv for _, kv in lens), sum(4 * -(-kv // c["page"]) for _, kv in lens)
    if c["op"] == "read":
        return {"bytes": 2 * keys * (code + c["hkv"] * c["D"] * BYTES[c["x"]]) + entries, "flops": 0}
    live = pairs = 0
    for n, kv in lens:
        w = c["window"] or kv
        live += min(kv, n - 1 + w)
        pairs += sum(min(w, kv - n + i + 1) for i in range(n))
    return {"bytes": 2 * live * code + T * c["hq"] * (c["D"] * 4 + 4) + entries, "flops": 4 * c["D"] * c["hq"] * pairs}


# ------------------------------------------------------------------ the definitions in 64 bits

def exact(case, seed):
    c = dict(case)
    s = prepare(c, seed)
    return {"append": _exact_append, "read": _exact_read, "attn": _exact_attn, "linear": _exact_linear}[c["op"]](c, s)


def _slots(c, s, b, lo, hi):
    """Page and slot of the keys lo .. hi of sequence b."""
    j = torch.arange(lo, hi, device="cuda")
    return s["table"][b].long()[j // c["page"]], j % c["page"]


def _codes64(c, z):
    if c["fmt"] == "e4m3":
        return z.float().clamp(-448, 448).to(torch.float8_e4m3fn)
    return torch.trunc(z + torch.copysign(torch.full_like(z, 0.5), z))


def _exact_append(c, s):
    r, at = {}, 0
    vals = {n: s[n + "c"].double() * s[n + "s"].double().unsqueeze(-1) if c["fmt"] == "int8" else s[n + "c"].clone()
            for n in ("k", "v")}
    scales = {n: s[n + "s"].double() for n in ("k", "v")}
    for b, (n, kv) in enumerate(s["lens"]):
        page, slot = _slots(c, s, b, kv - n, kv)
        for name in ("k", "v"):
            x = s[name + "n"][at:at + n].double()
            d = torch.linalg.vector_norm(x, ord=math.inf, dim=2) / TOP[c["fmt"]]
            z = torch.nan_to_num(x / d.unsqueeze(2), nan=0.0)
            codes = _codes64(c, z)
            scales[name][page, slot] = d
            if c["fmt"] == "int8":
                vals[name][page, slot] = codes * d.unsqueeze(2)
            else:
                vals[name].view(torch.uint8)[page, slot] = codes.view(torch.uint8)
        at += n
    for name in ("k", "v"):
        r[name + "s"] = scales[name]
    for name in ("k", "v"):
        r[name] = vals[name].double()
    return r


def _exact_read(c, s):
    r = {}
    for name in ("k", "v"):
        out = s[name + "o"].double()
        for b, (_, kv) in enumerate(s["lens"]):
            page, slot = _slots(c, s, b, 0, kv)
            lo = int(s["first"][b])
            part = s[name + "c"].view(torch.uint8)[page, slot].view(s[name + "c"].dtype).double()
            out[lo:lo + kv] = part * s[name + "s"][page, slot].double()[:, :, None]
        r[name] = out
    return r


def _exact_attn(c, s):
    hq, hkv, D = c["hq"], c["hkv"], c["D"]
    G, T = hq // hkv, s["qn"].shape[0]
    out = torch.empty((T, hq, D), dtype=torch.float64, device="cuda")
    lse = torch.empty((T, hq), dtype=torch.float64, device="cuda")
    at = 0
    for b, (n, kv) in enumerate(s["lens"]):
        page, slot = _slots(c, s, b, 0, kv)
        pos = torch.arange(kv - n, kv, device="cuda")[:, None]
        j = torch.arange(kv, device="cuda")[None]
        hidden = j > pos
        if c["window"]:
            hidden = hidden | (pos - j >= c["window"])
        hidden = hidden.repeat_interleave(G, 0)
        for h in range(hkv):
            key = s["kc"].view(torch.uint8)[page, slot, h].view(s["kc"].dtype).double()
            val = s["vc"].view(torch.uint8)[page, slot, h].view(s["vc"].dtype).double()
            q = s["qn"][at:at + n, h * G:(h + 1) * G].double().reshape(n * G, D)
            a = q @ key.T * s["ks"][page, slot, h].double() * s["scale"]
            a = a.masked_fill(hidden, -math.inf)
            p = torch.softmax(a, 1) * s["vs"][page, slot, h].double()
            out[at:at + n, h * G:(h + 1) * G] = (p @ val).view(n, G, D)
            lse[at:at + n, h * G:(h + 1) * G] = torch.logsumexp(a, 1).view(n, G)
        at += n
    return {"out": out, "lse": lse}


def _exact_linear(c, s):
    y = torch.addmm(s["bias"].double() if s["bias"] is not None else torch.zeros(1, dtype=torch.float64, device="cuda"),
                    s["x"].double(), s["w"].double().T)
    f = torch.nn.functional
    y = {"none": lambda t: t, "relu": torch.relu, "silu": f.silu, "gelu": f.gelu,
         "gelu_tanh": lambda t: f.gelu(t, approximate="tanh")}[c["act"]](y)
    return {"out": y if s["res"] is None else y + s["res"].double()}
