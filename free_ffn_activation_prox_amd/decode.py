"""Decode-step harness: a random-weight, Llama-shaped decoder whose FFNs run
either dense or through the Prox library, to put the FFN speed-up next to the
end-to-end decode step ("Prox: ...", Abstract, reports 1.99x end-to-end at
70 % FFN sparsity; "PrunePath: ...", §4.5: the parts other than the FFN cap
the end-to-end gain).

Everything but the FFN is the unchanged decoder block, in torch on the GPU:
pre-norm RMSNorm (eps 1e-5), q/k/v/o projections (bf16, nn.Linear layout; q,
k and v as one product), rotary embedding (theta 10000, pairs (2i, 2i + 1),
one complex product for q and one for k, the attention scale 1/sqrt(head_dim)
folded into q's), attention over a bf16 KV cache, residuals, written with few
kernels so that the step is not dominated by launches of tiny ones.  The FFN
is one of:
  "dense"  the SwiGLU FFN as three bf16 matrix products (torch / hipBLASLt);
  "prox"   prox_ffn_forward (a proxy kind, k_in, k_ff);
  "q8"     prox_ffn_forward_q8 (int8 Stage-2 rows);
  "exact"  the exact-mask mode.
One step = one token through every layer, at the next cache position.

With cache "int8" or "fp8" the harness keeps its keys and values in the paged
8-bit cache instead: norm of q and k where a layer has gains for it, rotation
and append in one call, attention over the pages in another, for one or more
sequences, and prompts (``prefill``) besides single tokens.  The sequences'
lengths are kept on the device, so a captured step goes on by a token with
every replay.
"""

from __future__ import annotations

import math
from dataclasses import dataclass
from typing import List, Optional

import numpy as np
import torch

from . import (KV_PAGE, KVBatch, KVCache, Weights, alloc_kv_workspace, alloc_workspace, build_proxy, build_qweights,
               ffn_forward, kv_append, kv_attention)

EPS = 1e-5
THETA = 10000.0
MAX_PREFILL = 4096     # tokens of one pass through the layers (PROX_MAX_BATCH)


@dataclass
class DecoderShape:
    n_layers: int
    d: int
    F: int
    n_heads: int
    n_kv: int

    @property
    def hd(self) -> int:
        return self.d // self.n_heads


class DecodeHarness:
    """Decode steps of a stack of decoder layers with bf16 weights.

    ``layers``: per layer a dict of bf16 device tensors wq [d][d],
    wk, wv [n_kv * hd][d], wo [d][d], g_attn, g_ffn [d], wg_t, wu_t, wd [F][d]
    (wd row j = W_down[j, :]).  ``ffn``: "dense" | "prox" | "q8" | "exact".
    ``cache``: "dense" (bf16, one sequence) or the paged 8-bit cache, "int8" |
    "fp8", of ``n_seq`` sequences; layers may then have g_q, g_k [hd], the gains
    of a norm of every head of q and k before the rotation."""

    def __init__(self, shape: DecoderShape, layers: List[dict], max_ctx: int, ffn: str = "prox",
                 proxy: str = "int8", k_in: Optional[int] = None, k_ff: Optional[int] = None, device="cuda",
                 cache: str = "dense", n_seq: int = 1):
        if cache == "dense" and (n_seq != 1 or any("g_q" in L or "g_k" in L for L in layers)):
            raise ValueError("the dense cache holds one sequence and has no norm of q and k: use cache='int8' or 'fp8'")
        self.cache, self.n_seq = cache, n_seq
        self.shape, self.layers, self.ffn = shape, layers, ffn
        self.max_ctx = max_ctx
        d, F, hd = shape.d, shape.F, shape.hd
        self.k_in = d if ffn == "exact" else (k_in if k_in is not None else d)
        self.k_ff = k_ff if k_ff is not None else F
        # q, k and v projections as one product (rows of wq, wk, wv stacked)
        self.wqkv = [torch.cat([L["wq"], L["wk"], L["wv"]], 0).contiguous() for L in layers]
        # rotary factors e^{i pos theta^(-2i/hd)} per position; the query's
        # carry the attention scale 1/sqrt(hd)
        n_pages = -(-max_ctx // KV_PAGE)
        i = torch.arange(hd // 2, dtype=torch.float64)
        ang = torch.arange(max_ctx if cache == "dense" else n_pages * KV_PAGE, dtype=torch.float64)[:, None] * (THETA ** (-2.0 * i / hd))[None, :]
        rot = torch.polar(torch.ones_like(ang), ang)
        self.rot_k = rot.to(torch.complex64).to(device)
        self.rot_q = (rot / math.sqrt(hd)).to(torch.complex64).to(device)
        self.g_attn = [L["g_attn"].float() for L in layers]
        self.g_ffn = [L["g_ffn"].float() for L in layers]
        if cache == "dense":
            # K cache stored transposed ([kv][hd][ctx]) so q.K is a product with a
            # row-major right operand; V cache [kv][ctx][hd]
            self.Kt = [torch.zeros(shape.n_kv, hd, max_ctx, dtype=torch.bfloat16, device=device) for _ in layers]
            self.V = [torch.zeros(shape.n_kv, max_ctx, hd, dtype=torch.bfloat16, device=device) for _ in layers]
        else:
            self.kv = [KVCache.alloc(cache, n_seq * n_pages, shape.n_kv, hd, device) for _ in layers]
            dev = self.kv[0].device
            self.g_q = [L["g_q"].float() if "g_q" in L else None for L in layers]
            self.g_k = [L["g_k"].float() if "g_k" in L else None for L in layers]
            self.table = torch.arange(n_seq * n_pages, dtype=torch.int32, device=dev).view(n_seq, n_pages)
            self.ctx = torch.zeros(n_seq, dtype=torch.int32, device=dev)   # tokens of each sequence
            self.lengths = [0] * n_seq           # the same on the host (a replayed graph does not move it)
            self.one = KVBatch(self.ctx, self.table)
            self.kv_ws = alloc_kv_workspace(self.kv[0], self.one, shape.n_heads)
        self.pos = 0
        if ffn != "dense":
            kind = "exact" if ffn == "exact" else proxy
            self.w = [Weights(L["wg_t"], L["wu_t"], L["wd"]) for L in layers]
            self.px = [build_proxy(w, kind) for w in self.w]
            self.s2 = [build_qweights(w) for w in self.w] if ffn == "q8" else self.w
            self.ws = alloc_workspace(d, F, n_seq, kind, device)
            self.y = torch.empty(n_seq, d, dtype=torch.float32, device=device)
            self.mask = torch.empty(n_seq, F, dtype=torch.uint8, device=device)
            self.idx = torch.empty(n_seq, max(self.k_ff, 1), dtype=torch.int32, device=device)
        self.taps: Optional[dict] = None

    def fill_cache(self, n: int, seed: int = 0):
        """Random keys and values at positions 0..n-1 (a context of n tokens, of every sequence)."""
        g = torch.Generator(device="cpu").manual_seed(seed)
        if self.cache != "dense":
            if n > self.max_ctx:
                raise ValueError(f"{n} tokens do not fit the cache's {self.max_ctx} positions")
            self.lengths = [0] * self.n_seq
            self._grow(range(self.n_seq), n)
            self.ctx.fill_(n)
            T = self.n_seq * n
            start = torch.arange(0, T + 1, n, dtype=torch.int32, device=self.ctx.device) if n else torch.zeros_like(self.ctx)
            batch = KVBatch(self.ctx, self.table, start, n_tokens=T, max_q=n) if n else None
            for kv in self.kv if n else ():
                k, v = (torch.randn(T, kv.n_kv, kv.head_dim, generator=g).to(torch.bfloat16).to(kv.device) for _ in range(2))
                kv_append(kv, batch, k, v)
            return
        for Kt, V in zip(self.Kt, self.V):
            Kt[:, :, :n] = torch.randn(Kt[:, :, :n].shape, generator=g).to(Kt.dtype).to(Kt.device)
            V[:, :n, :] = torch.randn(V[:, :n, :].shape, generator=g).to(V.dtype).to(V.device)
        self.pos = n

    def _rmsnorm(self, x, g):
        return torch.nn.functional.rms_norm(x, (x.shape[-1],), g, EPS).to(torch.bfloat16)

    def _ffn(self, li: int, f_in: torch.Tensor) -> torch.Tensor:
        L = self.layers[li]
        if self.ffn == "dense":
            g = torch.nn.functional.linear(f_in, L["wg_t"])
            u = torch.nn.functional.linear(f_in, L["wu_t"])
            h = (torch.nn.functional.silu(g.float()) * u.float()).to(torch.bfloat16)
            return torch.matmul(h, L["wd"]).float()
        if f_in.shape[0] != self.y.shape[0]:                  # a prompt
            return ffn_forward(f_in, self.s2[li], self.px[li], self.k_in, self.k_ff)[0]
        ffn_forward(f_in, self.s2[li], self.px[li], self.k_in, self.k_ff, y=self.y, mask=self.mask, idx=self.idx,
                    workspace=self.ws)
        return self.y

    def _grow(self, seqs, n: int):
        """n more tokens of the sequences `seqs`, on the host's count."""
        if max(self.lengths[s] for s in seqs) + n > self.max_ctx:
            raise ValueError(f"{n} more tokens do not fit the cache's {self.max_ctx} positions")
        for s in seqs:
            self.lengths[s] += n
        self.pos = max(self.lengths)

    def _paged(self, x: torch.Tensor, batch: KVBatch, workspace) -> torch.Tensor:
        """x fp32 [rows][d], the batch's rows, through every layer over the paged cache."""
        sh = self.shape
        H, KV, hd, d, T = sh.n_heads, sh.n_kv, sh.hd, sh.d, x.shape[0]
        for li, L in enumerate(self.layers):
            a = self._rmsnorm(x, self.g_attn[li])
            qkv = torch.nn.functional.linear(a, self.wqkv[li]).view(T, H + 2 * KV, hd)
            q, k, v = qkv.split([H, KV, KV], 1)
            q = kv_append(self.kv[li], batch, k, v, rot=self.rot_k, q=q, g_q=self.g_q[li], g_k=self.g_k[li], eps=EPS)
            att = kv_attention(q, self.kv[li], batch, workspace=workspace)
            x = x + torch.nn.functional.linear(att.view(T, d), L["wo"])
            f_in = self._rmsnorm(x, self.g_ffn[li])
            f_out = self._ffn(li, f_in)
            if self.taps is not None:
                for n, t in (("attn_in", a), ("x_mid", x), ("ffn_in", f_in), ("ffn_out", f_out)):
                    self.taps.setdefault(n, []).append(t.clone())
            x = x + f_out
        return x

    def prefill(self, x: torch.Tensor, seq: int = 0) -> torch.Tensor:
        """The next tokens of one sequence, x fp32 [tokens][d], through every
        layer (up to 4096 at a time); paged cache only."""
        if self.cache == "dense":
            raise ValueError("prefill needs the paged cache (cache='int8' or 'fp8')")
        if not 0 <= seq < self.n_seq:
            raise ValueError(f"sequence {seq} of {self.n_seq}")
        if x.dim() != 2 or x.shape[1] != self.shape.d:
            raise ValueError("x must be [tokens][d]")
        self._grow([seq], x.shape[0])
        out = []
        for p in x.split(MAX_PREFILL) if x.shape[0] else ():
            T = p.shape[0]
            self.ctx[seq:seq + 1].add_(T)
            start = torch.tensor([0, T], dtype=torch.int32, device=self.ctx.device)
            batch = KVBatch(self.ctx[seq:seq + 1], self.table[seq:seq + 1], start, n_tokens=T, max_q=T)
            out.append(self._paged(p, batch, alloc_kv_workspace(self.kv[0], batch, self.shape.n_heads)))
        return torch.cat(out) if out else x

    def step(self, x: torch.Tensor) -> torch.Tensor:
        """x fp32 [n_seq][d] -> fp32 [n_seq][d] after every layer; the cache advances."""
        if self.cache != "dense":
            if x.shape != (self.n_seq, self.shape.d):
                raise ValueError("x must be [n_seq][d]")
            self._grow(range(self.n_seq), 1)
            self.ctx.add_(1)
            return self._paged(x, self.one, self.kv_ws)
        sh, pos = self.shape, self.pos
        H, KV, hd = sh.n_heads, sh.n_kv, sh.hd
        d, kvd = sh.d, sh.n_kv * sh.hd
        rep = H // KV
        T = pos + 1
        for li, L in enumerate(self.layers):
            a = self._rmsnorm(x, self.g_attn[li])
            qkv = torch.nn.functional.linear(a, self.wqkv[li])                     # [1][d + 2 kvd] bf16
            qk = torch.view_as_complex(qkv[0, :d + kvd].float().view(H + KV, hd // 2, 2))
            q = torch.view_as_real(qk[:H] * self.rot_q[pos]).to(torch.bfloat16).view(KV, rep, hd)
            self.Kt[li][:, :, pos].copy_(torch.view_as_real(qk[H:] * self.rot_k[pos]).view(KV, hd))
            self.V[li][:, pos, :].copy_(qkv[0, d + kvd:].view(KV, hd))
            sc = torch.matmul(q, self.Kt[li][:, :, :T])                          # heads grouped by kv head
            p = torch.softmax(sc, dim=-1, dtype=torch.float32).to(torch.bfloat16)
            att = torch.matmul(p, self.V[li][:, :T, :]).reshape(1, d)
            x = x + torch.nn.functional.linear(att, L["wo"])
            f_in = self._rmsnorm(x, self.g_ffn[li])
            f_out = self._ffn(li, f_in)
            if self.taps is not None:
                self.taps.setdefault("ffn_in", []).append(f_in.clone())
                self.taps.setdefault("ffn_out", []).append(f_out.clone())
                self.taps.setdefault("attn_in", []).append(a.clone())
                self.taps.setdefault("x_mid", []).append(x.clone())
                if self.ffn != "dense":
                    self.taps.setdefault("mask", []).append(self.mask.clone())
            x = x + f_out
        self.pos += 1
        return x


def random_layers(shape: DecoderShape, ffn_weights, seed: int = 0, device="cuda", std: float = 0.02):
    """Random bf16 decoder weights: attention N(0, std); FFN weights from
    ``ffn_weights(layer)`` (bf16 bit arrays wg_t, wu_t, wd [F][d]); RMSNorm
    gains 1."""
    d, kvd = shape.d, shape.n_kv * shape.hd
    g = torch.Generator(device="cpu").manual_seed(seed)

    def rnd(*s):
        return (torch.randn(s, generator=g) * std).to(torch.bfloat16).to(device)

    def bits(a):
        return torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16).to(device)

    out = []
    for li in range(shape.n_layers):
        w = ffn_weights(li)
        out.append({"wq": rnd(d, d), "wk": rnd(kvd, d), "wv": rnd(kvd, d), "wo": rnd(d, d),
                    "g_attn": torch.ones(d, dtype=torch.bfloat16, device=device),
                    "g_ffn": torch.ones(d, dtype=torch.bfloat16, device=device),
                    "wg_t": bits(w["wg_t"]), "wu_t": bits(w["wu_t"]), "wd": bits(w["wd"])})
    return out
