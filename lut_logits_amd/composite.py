"""A per-token decode loop over the compressed parts of a Gemma-2-2B-shaped model, built from the
library's entry points: the current token's embedding row (rq_decode_rows, fp32, times sqrt(D) as
Gemma scales its embeddings), the MLP blocks (rq_lut_mlp) on a residual stream, and the tied head on
the last hidden vector (rq_build_lut + rq_lut_logits: softcap and argmax, no logits written). The
argmax id stays on the device and is the next token's row id, so a run of tokens is enqueued with no
host synchronisation.

Around each block sits Gemma-2's own glue, outside the method: an RMSNorm before the block and one
after it, the block's output added to the residual stream, and a final RMSNorm before the head. One
rq_residual_norm launch per block does it (h += rms(y), then the next input rms(h)). The norms carry
unit scales (Gemma-2 stores each RMSNorm scale as 1 + w, and w starts at zero). Without them the chain diverges on these synthetic weights: a block maps an input of
scale s to about 1.3 s^2, so an unnormalised chain of 26 blocks overflows fp32 within ten.

Attention is part of the loop where the caller has its projections (AttentionBlock: in 4 bits, as the combined RQ+NF4
variant keeps them): four calls a layer (rq_q4_matvec, rq_rope_append, rq_paged_attn, rq_q4_matvec) in the same glue, on a
paged cache that the loop keeps; the token's place is read on the device like its id."""
import math

import torch

from . import binding as B
from .rotary import rope_freqs

RMS_EPS = 1e-6


class AttentionBlock:
    """One layer's attention with 4-bit projections (Q4Matrix): qkv [(heads + 2 kv_heads) * size][D] stacks the rows of q, k and
    v; out [D][heads * size]. window: sliding window in tokens (0: none), which Gemma-2 has in every other layer."""

    def __init__(self, qkv, out, heads, kv_heads, size, window=0):
        if heads % kv_heads:
            raise ValueError(f"heads={heads} is no multiple of kv_heads={kv_heads}")
        if qkv.rows != (heads + 2 * kv_heads) * size or out.D != heads * size or out.rows != qkv.D:
            raise ValueError(f"projections {qkv.rows} x {qkv.D} and {out.rows} x {out.D} do not fit {heads} + 2 x {kv_heads} "
                             f"heads of {size}")
        self.qkv, self.out, self.heads, self.kv_heads, self.size, self.window = qkv, out, heads, kv_heads, size, window


class DecodeLoop:
    """head: DeviceMatrix of the tied embedding / head; layers: list of (gate, up, down) DeviceMatrix; attention: None, or
    an AttentionBlock for each layer."""

    def __init__(self, head, layers, softcap=30.0, max_tokens=128, device="cuda", keep_layers=False, attention=None,
                 rope_base=10000.0, attn_softcap=50.0, page_size=16, cache_dtype=torch.bfloat16):
        """keep_layers: keep every block's input (ins[i], after the pre-norm) and output (outs[i]) of
        the last step, instead of one buffer each (attention: att_ins, att_qkv, att_q, att_mid, att_outs)."""
        self.head, self.layers, self.softcap = head, list(layers), softcap
        self.scale = math.sqrt(head.D)
        self.ids = torch.zeros(max_tokens + 1, dtype=torch.int32, device=device)
        D = head.D

        def buf():
            return torch.empty((1, D), dtype=torch.float32, device=device)

        self.row = buf()
        self.h = buf()       # residual stream
        self.last = buf()    # final-norm output: the head's hidden vector
        n = len(self.layers) if keep_layers else 1
        self.ins = [buf() for _ in range(n)]
        self.outs = [buf() for _ in range(n)]
        self.attention = list(attention or [])
        if self.attention:
            self._init_attention(max_tokens, device, n, rope_base, attn_softcap, page_size, cache_dtype)
        self.lut = torch.empty(B.lut_bytes(head, 1) // 4, dtype=torch.float32, device=device)
        mlp_ws = max([B.lut_mlp_workspace(*lay, 1) for lay in self.layers] + [256])
        self.ws_mlp = B.workspace(mlp_ws, device)
        self.ws_head = B.workspace(B.lut_logits_workspace(head, 1), device)

    def _init_attention(self, max_tokens, device, n, base, softcap, page_size, dtype):
        if len(self.attention) != len(self.layers):
            raise ValueError(f"{len(self.attention)} attention blocks for {len(self.layers)} layers")
        first = self.attention[0]
        for a in self.attention:
            if a.qkv.D != self.head.D or (a.heads, a.kv_heads, a.size) != (first.heads, first.kv_heads, first.size):
                raise ValueError("attention blocks of different shapes, or not of the head's width")

        def buf(*shape, dt=torch.float32):
            return [torch.empty(shape, dtype=dt, device=device) for _ in range(n)]

        D, heads, kv, size = self.head.D, first.heads, first.kv_heads, first.size
        self.att_ins, self.att_outs = buf(1, D), buf(1, D)
        self.att_qkv = buf(1, (heads + 2 * kv) * size)
        self.att_q, self.att_mid = buf(1, heads, size, dt=dtype), buf(1, heads, size, dt=dtype)
        pages = -(-max_tokens // page_size)
        self.caches = [B.KVCache.empty(pages, kv, page_size, size, dtype, device) for _ in self.attention]
        self.cu_q = torch.tensor([0, 1], dtype=torch.int32, device=device)
        self.table = torch.arange(pages, dtype=torch.int32, device=device).view(1, pages)
        self.lens = torch.arange(1, max_tokens + 1, dtype=torch.int32, device=device)   # lens[t:t+1]: the length at token t
        self.freqs, _ = rope_freqs(size, base, device=device)
        self.max_len, self.attn_softcap = max_tokens, softcap
        self.ws_attn = B.workspace(B.paged_attn_workspace(self.caches[0], 1, 1, heads, max_tokens), device)

    def _attend(self, i, t):
        """Layer i's attention at token t: from its input to its output buffer (returned)."""
        a, j = self.attention[i], i % len(self.att_ins)
        heads, kv, size = a.heads, a.kv_heads, a.size
        row = B.q4_matvec(a.qkv, self.att_ins[j], out=self.att_qkv[j]).view(1, heads + 2 * kv, size)
        where = (self.caches[i], self.cu_q, self.lens[t:t + 1], self.table)
        B.rope_append(row[:, :heads], row[:, heads:heads + kv], row[:, heads + kv:], *where, self.freqs, out=self.att_q[j])
        B.paged_attn(self.att_q[j], *where, softcap=self.attn_softcap, window=a.window, max_len=self.max_len, ws=self.ws_attn,
                     out=self.att_mid[j])
        return B.q4_matvec(a.out, self.att_mid[j].view(1, heads * size), out=self.att_outs[j])

    def step(self, t):
        """Token t: row of ids[t] -> blocks on the residual stream -> final norm -> head argmax into
        ids[t + 1]. Returns the head's hidden vector."""
        B.decode_rows(self.head, self.ids[t:t + 1], "f32", out=self.row)
        torch.mul(self.row, self.scale, out=self.h)
        n = len(self.layers)

        def block_input(i):   # block i's input buffer; past the last block, the head's vector
            return self.ins[i % len(self.ins)] if i < n else self.last

        def layer_input(i):   # where layer i begins: with its attention, if it has one
            return self.att_ins[i % len(self.att_ins)] if self.attention and i < n else block_input(i)

        B.residual_norm(self.h, layer_input(0), eps=RMS_EPS)
        for i, (gate, up, down) in enumerate(self.layers):
            if self.attention:
                B.residual_norm(self.h, block_input(i), self._attend(i, t), eps=RMS_EPS)
            y = self.outs[i % len(self.outs)]
            B.lut_mlp(gate, up, down, block_input(i), ws=self.ws_mlp, out=y)
            B.residual_norm(self.h, layer_input(i + 1), y, eps=RMS_EPS)
        B.build_lut(self.head, self.last, out=self.lut)
        B.lut_logits(self.head, self.lut, 1, softcap=self.softcap, logits=False, ws=self.ws_head,
                     argmax_out=self.ids[t + 1:t + 2])
        return self.last

    def run(self, first_id, n_tokens):
        """Enqueue n_tokens steps starting from token first_id; the ids are in self.ids[:n_tokens + 1]."""
        self.ids[0] = int(first_id)
        for t in range(n_tokens):
            self.step(t)
        return self.ids[:n_tokens + 1]
