"""A decoder block around the MoE layer: the operators of this package run together, as a serving step uses them.

    y      = norm(x)                                   moe_add_rmsnorm
    q,k,v  = y Wqkv  [, rotary embedding]              torch matmul or moe_linear, the caller's function
    cache += k, v                                      moe_kv_append or moe_kv_append_q8
    o      = attention(q, cache) Wo                    moe_paged_attention or _q8, torch matmul or moe_linear
    r      = x + o,  z = norm(r),  codes = q8_K(z)     moe_add_rmsnorm
    logits = z Wr;  ids, gates = route(logits)         torch matmul in fp32, moe_route_grouped
    out    = r + sum of the experts' outputs           moe_bucket, moe_expert_ffn, moe_combine

A call takes any mixture of sequences (single tokens, drafts to verify, prompt chunks) over one paged cache.  The
residual stream is fp32, attention runs in the cache's type, the experts on q8_K codes.  Everything is launched on the
current stream into buffers of the block, so a step can be captured into a CUDA graph.

With `fused` (or with biases) the projections run on moe_linear, which adds the attention's output to the fp32 residual
stream unrounded.  A cache of 8-bit codes (`q8_cache`, with scales) is quantised as it is written and read as it lies;
prompt chunks read it back into `read_rows` rows of the block first, where the 16-bit attention is several times faster
on many rows.
"""
from __future__ import annotations

import block_quantized_routed_gb300 as moe


READ_PAGE = 64   # keys of a page of the rows that an 8-bit cache is read back into
# It is for more new tokens per sequence, on average, than this.  Over the codes / by way of 16 bits, in us, every sequence
# with 4 / 8 / 16 new tokens: 16 of 4096 keys (32 heads over 4 of 128) 43/74, 66/75, 115/77; 2 of 8192 35/28, 37/29, 44/31;
# 1 of 65536 (64 over 8) 84/125, 117/126, 206/128; 8 of 4096 (40 over 8 of 64) 29/46, 44/51, 60/51; 4 of 4096 (16 over 2 of
# 256) 25/29, 31/30, 39/34.  One rule for the call: a long chunk among single tokens takes their caches with it.
READ_FROM = 8


def _tf32(torch):
    """Whether the caller's settings let fp32 matrix products run in TF32.  Router logits must not: its 2^-11 would
    change choices, so the layer's own router forms them then."""
    matmul = torch.backends.cuda.matmul
    if not hasattr(matmul, "fp32_precision"):
        return matmul.allow_tf32
    own = matmul.fp32_precision
    return (torch.backends.fp32_precision if own == "none" else own) == "tf32"


class MoeDecoderBlock:
    """One block's weights, buffers for up to desc.T_max tokens, and forward().

    desc: MoE layer descriptor (H, I, E, top_k, n_shared, route, fmt, T_max); table: its expert_table;
    w_qkv [(Hq + 2 Hkv) D, H] and w_o [H, Hq D] in the cache's type; norms fp32 [H]; w_router fp32 [E, H];
    router_bias fp32 [E] or None takes part in the selection only.  n_group, topk_group, group_score, renorm and
    scale are moe_route_grouped's; rotary(q, k, cu_q, kv_len) rotates the views q [T, Hq, D] and k [T, Hkv, D] in
    place; window > 0 limits attention to the last keys.  fused: the projections by moe_linear; b_qkv fp32 and b_o fp32,
    their biases, ask for it too.  q8_cache: forward() may be given 8-bit caches; read_rows: rows of 16 bits for reading
    them back (a call's sequences take whole runs of 64 rows each), 0 to attend to the codes always.
    """

    def __init__(self, desc, table, attn_norm, w_qkv, w_o, ffn_norm, w_router, n_heads, n_kv_heads, head_dim,
                 router_bias=None, n_group=1, topk_group=1, group_score=moe.GROUP_TOP2, renorm=True, scale=1.0,
                 eps=1e-6, window=0, rotary=None, device="cuda", b_qkv=None, b_o=None, fused=False, q8_cache=False,
                 read_rows=0):
        import torch
        self.desc = d = moe._desc(desc)
        if w_router.shape != (d.E, d.H) or w_router.dtype != torch.float32:
            raise moe.MoeError(moe.MOE_ERR_INVALID_ARG, "MoeDecoderBlock: w_router must be fp32 [E, H]")
        self.table, self.attn_norm, self.w_qkv, self.w_o = table, attn_norm, w_qkv, w_o
        self.ffn_norm, self.w_router, self.router_bias = ffn_norm, w_router.contiguous(), router_bias
        self.heads, self.kv_heads, self.head_dim = n_heads, n_kv_heads, head_dim
        self.routing = dict(route=d.route, n_group=n_group, topk_group=topk_group, group_score=group_score,
                            renorm=renorm, scale=scale)
        self.eps, self.window, self.rotary = eps, window, rotary
        T, H, k, S, E = d.T_max, d.H, d.top_k, d.n_shared, d.E
        attn_ws = moe.moe_paged_attention_workspace_size(n_heads, n_kv_heads, head_dim)
        ffn_ws = moe.moe_expert_ffn_workspace_size(d, T)
        if attn_ws == 0 or ffn_ws == 0:
            raise moe.MoeError(moe.MOE_ERR_UNSUPPORTED, "MoeDecoderBlock")
        new = lambda *shape, dtype=torch.float32: torch.empty(shape, dtype=dtype, device=device)
        act = w_qkv.dtype
        self.y = new(T, H, dtype=act)
        self.qkv = new(T, (n_heads + 2 * n_kv_heads) * head_dim, dtype=act)
        self.attn = new(T, n_heads * head_dim, dtype=act)
        self.o = new(T, H, dtype=act)
        self.resid, self.z = new(T, H), new(T, H)
        self.q = new(T, H, dtype=torch.int8)
        self.d = new(T, H // 256)
        self.bsum16 = new(T, H // 16, dtype=torch.int16)
        self.logits = new(T, E)
        self.ids, self.gates = new(T, k, dtype=torch.int32), new(T, k)
        self.counts, self.offsets = new(E + S, dtype=torch.int32), new(E + S + 1, dtype=torch.int32)
        self.perm = new(T * (k + S), dtype=torch.int32)
        self.y_slots = new(T * (k + S), H)
        zeros = lambda n: torch.zeros(n, dtype=torch.uint8, device=device)
        self.attn_ws, self.ffn_ws = zeros(attn_ws), zeros(ffn_ws)
        self.bucket_ws = zeros(moe.moe_bucket_workspace_size(T, k, E, S))
        self.b_qkv, self.b_o, self.fused = b_qkv, b_o, fused or b_qkv is not None or b_o is not None
        self.q8_ws = self.k_read = self.v_read = None
        if q8_cache:
            self.q8_ws = zeros(moe.moe_paged_attention_q8_workspace_size(n_heads, n_kv_heads, head_dim))
            if read_rows:
                pages = -(-read_rows // READ_PAGE)
                self.k_read, self.v_read = (new(pages * READ_PAGE, n_kv_heads, head_dim, dtype=act) for _ in range(2))

    def _attend_q8(self, q, k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_q, kv_len, attn):
        """Appends to an 8-bit cache and attends to it."""
        import torch
        T, n_seqs, D = q.shape[0], kv_len.shape[0], self.head_dim
        moe.moe_kv_append_q8(k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_q, kv_len, self.q8_ws)
        if self.k_read is None or T <= READ_FROM * n_seqs:
            moe.moe_paged_attention_q8(q, k_cache, v_cache, k_scale, v_scale, page_table, cu_q, kv_len, D ** -0.5, attn,
                                       self.q8_ws, window=self.window)
            return
        # the sequences one after another in whole pages; lengths are known on the device only
        runs = (kv_len.clamp(min=0) + (READ_PAGE - 1)) // READ_PAGE
        first = (torch.cumsum(runs, 0) - runs).to(torch.int32)
        most = -(-page_table.shape[1] * k_cache.shape[1] // READ_PAGE)
        table = (first.unsqueeze(1) + torch.arange(most, dtype=torch.int32, device=q.device)).to(torch.int32)
        moe.moe_kv_read_q8(k_cache, v_cache, k_scale, v_scale, page_table, kv_len, first * READ_PAGE, self.k_read,
                           self.v_read, self.q8_ws)
        pages = lambda t: t.view(-1, READ_PAGE, self.kv_heads, D)
        moe.moe_paged_attention(q, pages(self.k_read), pages(self.v_read), table, cu_q, kv_len, D ** -0.5, attn,
                                self.attn_ws, window=self.window)

    def forward(self, x, k_cache, v_cache, page_table, cu_q, kv_len, out=None, k_scale=None, v_scale=None):
        """x fp32 [T, H]: the residual stream of the call's new tokens, in the order of cu_q.  kv_len counts the new
        tokens.  k_scale and v_scale: of an 8-bit cache.  Returns out fp32 [T, H] (may be x; rows may have a stride)."""
        import torch
        T, d = x.shape[0], self.desc
        if T > d.T_max:
            raise moe.MoeError(moe.MOE_ERR_INVALID_ARG, "MoeDecoderBlock.forward: more tokens than T_max")
        if out is None:
            out = torch.empty(x.shape, dtype=torch.float32, device=x.device)
        elif out.shape != x.shape or out.dtype != torch.float32 or out.device != x.device:
            raise moe.MoeError(moe.MOE_ERR_INVALID_ARG, "MoeDecoderBlock.forward: out must be fp32 like x")
        if k_scale is not None and self.q8_ws is None:
            raise moe.MoeError(moe.MOE_ERR_INVALID_ARG, "MoeDecoderBlock.forward: an 8-bit cache needs q8_cache")
        if T == 0:
            return out
        hq, hkv, D = self.heads, self.kv_heads, self.head_dim
        y, qkv, attn, o, resid, z = (t[:T] for t in (self.y, self.qkv, self.attn, self.o, self.resid, self.z))
        moe.moe_add_rmsnorm(x, self.attn_norm, self.eps, y=y)
        if self.fused:
            moe.moe_linear(y, self.w_qkv, qkv, bias=self.b_qkv, ws=self.attn_ws)
        else:
            torch.matmul(y, self.w_qkv.t(), out=qkv)
        h = qkv.view(T, hq + 2 * hkv, D)
        q, k, v = h[:, :hq], h[:, hq:hq + hkv], h[:, hq + hkv:]
        if self.rotary is not None:
            self.rotary(q, k, cu_q, kv_len)
        if k_scale is not None:
            self._attend_q8(q, k, v, k_cache, v_cache, k_scale, v_scale, page_table, cu_q, kv_len, attn.view(T, hq, D))
        else:
            moe.moe_kv_append(k, v, k_cache, v_cache, page_table, cu_q, kv_len, self.attn_ws)
            moe.moe_paged_attention(q, k_cache, v_cache, page_table, cu_q, kv_len, D ** -0.5, attn.view(T, hq, D),
                                    self.attn_ws, window=self.window)
        q8, sc, bs = self.q[:T], self.d[:T], self.bsum16[:T]
        if self.fused:
            moe.moe_linear(attn, self.w_o, resid, bias=self.b_o, residual=x, ws=self.attn_ws)
            moe.moe_add_rmsnorm(resid, self.ffn_norm, self.eps, y=z, q_fmt=moe.NORM_Q_Q8K, q=q8, d=sc, bsum16=bs)
        else:
            torch.matmul(attn, self.w_o.t(), out=o)
            moe.moe_add_rmsnorm(o, self.ffn_norm, self.eps, residual=x, sum_out=resid, y=z, q_fmt=moe.NORM_Q_Q8K, q=q8,
                                d=sc, bsum16=bs)
        logits, ids, gates = self.logits[:T], self.ids[:T], self.gates[:T]
        if _tf32(torch):  # (as fast for long chunks alone: 64 tokens of 256 experts 227 us instead of 21)
            moe.moe_route_topk(z, self.w_router, None, d.top_k, d.route, logits, ids, gates)  # (its choices are not used)
        else:
            torch.matmul(z, self.w_router.t(), out=logits)
        moe.moe_route_grouped(logits, d.top_k, ids, gates, bias=self.router_bias, **self.routing)
        P = T * (d.top_k + d.n_shared)
        moe.moe_bucket(ids, d.E, d.n_shared, self.counts, self.offsets, self.perm, None, self.bucket_ws)
        moe.moe_expert_ffn(d, self.table, q8, sc, bs, self.counts, self.offsets, self.perm, T, self.y_slots[:P],
                           self.ffn_ws)
        # moe_combine takes rows without gaps on 16-byte boundaries
        rows = out if out.is_contiguous() and out.data_ptr() % 16 == 0 else torch.empty_like(resid)
        moe.moe_combine(self.y_slots[:P], gates, T, d.H, d.top_k, d.n_shared, resid, rows)
        if rows is not out:
            out.copy_(rows)
        return out

    def status(self):
        """Synchronises and returns the first device-recorded error since the last call (0: none).  The block can be used
        again after any of them: a wait that ran out leaves counters behind, which are cleared here."""
        import torch
        spaces = [ws for ws in (self.attn_ws, self.bucket_ws, self.ffn_ws, self.q8_ws) if ws is not None]
        found = [moe.moe_get_status(ws) for ws in spaces]
        for ws, st in zip(spaces, found):
            if st == moe.MOE_ERR_DEVICE_TIMEOUT and (ws is self.attn_ws or ws is self.q8_ws):
                ws.zero_()
                torch.cuda.current_stream().synchronize()
        return next((st for st in found if st != moe.MOE_OK), moe.MOE_OK)
