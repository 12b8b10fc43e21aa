"""A decoder block around the MoE layer: the operators of this package run together, as a serving step uses them.

    y      = norm(x)                                   moe_add_rmsnorm
    q,k,v  = y Wqkv  [, rotary embedding]              torch matmul, the caller's function
    cache += k, v                                      moe_kv_append
    o      = attention(q, cache) Wo                    moe_paged_attention, torch matmul
    r      = x + o,  z = norm(r),  codes = q8_K(z)     moe_add_rmsnorm
    logits = z Wr;  ids, gates = route(logits)         torch matmul in fp32, moe_route_grouped
    out    = r + sum of the experts' outputs           moe_bucket, moe_expert_ffn, moe_combine

A call takes any mixture of sequences (single tokens, drafts to verify, prompt chunks) over one paged cache.  The
residual stream is fp32, attention runs in the cache's type, the experts on q8_K codes.  Everything is launched on the
current stream into buffers of the block, so a step can be captured into a CUDA graph.
"""
from __future__ import annotations

import block_quantized_routed_gb300 as moe


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
    place; window > 0 limits attention to the last keys.
    """

    def __init__(self, desc, table, attn_norm, w_qkv, w_o, ffn_norm, w_router, n_heads, n_kv_heads, head_dim,
                 router_bias=None, n_group=1, topk_group=1, group_score=moe.GROUP_TOP2, renorm=True, scale=1.0,
                 eps=1e-6, window=0, rotary=None, device="cuda"):
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

    def forward(self, x, k_cache, v_cache, page_table, cu_q, kv_len, out=None):
        """x fp32 [T, H]: the residual stream of the call's new tokens, in the order of cu_q.  kv_len counts the new
        tokens.  Returns out fp32 [T, H] (may be x; rows may have a stride)."""
        import torch
        T, d = x.shape[0], self.desc
        if T > d.T_max:
            raise moe.MoeError(moe.MOE_ERR_INVALID_ARG, "MoeDecoderBlock.forward: more tokens than T_max")
        if out is None:
            out = torch.empty(x.shape, dtype=torch.float32, device=x.device)
        elif out.shape != x.shape or out.dtype != torch.float32 or out.device != x.device:
            raise moe.MoeError(moe.MOE_ERR_INVALID_ARG, "MoeDecoderBlock.forward: out must be fp32 like x")
        if T == 0:
            return out
        hq, hkv, D = self.heads, self.kv_heads, self.head_dim
        y, qkv, attn, o, resid, z = (t[:T] for t in (self.y, self.qkv, self.attn, self.o, self.resid, self.z))
        moe.moe_add_rmsnorm(x, self.attn_norm, self.eps, y=y)
        torch.matmul(y, self.w_qkv.t(), out=qkv)
        h = qkv.view(T, hq + 2 * hkv, D)
        q, k, v = h[:, :hq], h[:, hq:hq + hkv], h[:, hq + hkv:]
        if self.rotary is not None:
            self.rotary(q, k, cu_q, kv_len)
        moe.moe_kv_append(k, v, k_cache, v_cache, page_table, cu_q, kv_len, self.attn_ws)
        moe.moe_paged_attention(q, k_cache, v_cache, page_table, cu_q, kv_len, D ** -0.5, attn.view(T, hq, D),
                                self.attn_ws, window=self.window)
        torch.matmul(attn, self.w_o.t(), out=o)
        q8, sc, bs = self.q[:T], self.d[:T], self.bsum16[:T]
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
        found = [moe.moe_get_status(ws) for ws in (self.attn_ws, self.bucket_ws, self.ffn_ws)]
        if found[0] == moe.MOE_ERR_DEVICE_TIMEOUT:
            self.attn_ws.zero_()
            torch.cuda.current_stream().synchronize()
        return next((st for st in found if st != moe.MOE_OK), moe.MOE_OK)
