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

With keep_pages a step's attention reads that many pages of each sequence and
key head, those whose keys can give the largest scores by the bounds that the
harness keeps of every page (prompts see all pages).  With n_pages the sequences
take their pages from a pool of that many instead of each having its own share,
and may begin with a prompt in common (``share_prefix``): its pages are held once
and, where a step sees all pages, read once for all of them.  A sequence for which the pool has no page
left (``status`` [0] of them at the last step) keeps its tokens: the step's row is
behind them, where the table names no page, so it sees them and stores nothing
(past max_ctx it sees nothing either).  The host refuses what the pool cannot hold by its own
count, which replays do not move: a prompt looks at the device's once there is a
captured call, a step never waits for it.
"""

from __future__ import annotations

import math
from dataclasses import dataclass
from typing import List, Optional

import numpy as np
import torch

from . import (KV_PAGE, KVBatch, KVCache, KVPool, Weights, alloc_kv_bounds, alloc_kv_select_workspace,
               alloc_kv_selected_workspace, alloc_kv_shared_workspace, alloc_kv_workspace, alloc_workspace, build_proxy,
               build_qweights, ffn_forward, kv_append, kv_attention, kv_attention_selected, kv_attention_shared,
               kv_page_bounds, kv_pages, kv_select)

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
    of a norm of every head of q and k before the rotation.  ``keep_pages`` and
    ``n_pages`` (paged cache only): see above."""

    def __init__(self, shape: DecoderShape, layers: List[dict], max_ctx: int, ffn: str = "prox",
                 proxy: str = "int8", k_in: Optional[int] = None, k_ff: Optional[int] = None, device="cuda",
                 cache: str = "dense", n_seq: int = 1, keep_pages: Optional[int] = None,
                 n_pages: Optional[int] = None):
        if cache == "dense" and (keep_pages is not None or n_pages is not None):
            raise ValueError("keep_pages and n_pages need the paged cache (cache='int8' or 'fp8')")
        if keep_pages is not None and keep_pages < 2:
            raise ValueError("keep_pages must be at least 2: the first page and the last")
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
        width = -(-max_ctx // KV_PAGE)
        i = torch.arange(hd // 2, dtype=torch.float64)
        ang = torch.arange(max_ctx if cache == "dense" else width * KV_PAGE, dtype=torch.float64)[:, None] * (THETA ** (-2.0 * i / hd))[None, :]
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
            self.kv = [KVCache.alloc(cache, n_seq * width if n_pages is None else n_pages, shape.n_kv, hd, device) for _ in layers]
            dev = self.kv[0].device
            self.g_q = [L["g_q"].float() if "g_q" in L else None for L in layers]
            self.g_k = [L["g_k"].float() if "g_k" in L else None for L in layers]
            self.pool = None if n_pages is None else KVPool.alloc(n_pages, n_seq, width, dev)
            if self.pool is None:
                self.table = torch.arange(n_seq * width, dtype=torch.int32, device=dev).view(n_seq, width)
                self.ctx = torch.zeros(n_seq, dtype=torch.int32, device=dev)   # tokens of each sequence
            else:
                self.table, self.ctx = self.pool.block_table, self.pool.ctx_len
                self.want = torch.zeros_like(self.ctx)
                self.start = torch.zeros(n_seq + 1, dtype=torch.int32, device=dev)
                self.slots, self.status = torch.zeros_like(self.ctx), torch.zeros(2, dtype=torch.int32, device=dev)
            self.lengths = [0] * n_seq           # the same on the host (a replayed graph does not move it)
            self.captured = False                # whether a graph may have moved the pool's
            self.prefix = 0                      # pages that all sequences share
            # over a pool, rows of the tokens wanted: the lengths of all but the sequences that kv_pages refuses, whose
            # row is the first of a page that they do not have (by their lengths it would be their last token's again)
            self.one = KVBatch(self.ctx if self.pool is None else self.want, self.table)
            self.kv_ws = alloc_kv_workspace(self.kv[0], self.one, shape.n_heads)
            self.keep_pages = keep_pages
            if keep_pages is not None:
                self.bounds = [alloc_kv_bounds(kv) for kv in self.kv]
                self.picked = torch.empty(n_seq, shape.n_kv, keep_pages, dtype=torch.int32, device=dev)
                self.pick_ws = alloc_kv_select_workspace(self.kv[0], self.one, shape.n_heads)
                self.kv_ws = alloc_kv_selected_workspace(self.kv[0], self.one, shape.n_heads, keep_pages)
            if self.pool is not None:
                # these stay where they are: a captured step goes on using them when a prefix begins or ends
                self.shared = torch.zeros(1, dtype=torch.int32, device=dev)
                if keep_pages is None:
                    self.share_ws = alloc_kv_shared_workspace(self.kv[0], self.one, shape.n_heads)
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
            pages = self.n_seq * -(-n // KV_PAGE)
            if self.pool is not None and pages > self.pool.n_pages:
                raise ValueError(f"{self.n_seq} times {n} tokens need {pages} pages of a pool of {self.pool.n_pages}")
            self.lengths = [0] * self.n_seq
            if self.prefix:
                self.prefix = 0
                self.shared.zero_()
            self._grow(range(self.n_seq), n)
            T = self.n_seq * n
            if self.pool is None:
                self.ctx.fill_(n)
            else:
                kv_pages(self.pool, torch.zeros_like(self.ctx), 0)
                kv_pages(self.pool, torch.full_like(self.ctx, n), T)
            start = torch.arange(0, T + 1, n, dtype=torch.int32, device=self.ctx.device) if n else torch.zeros_like(self.ctx)
            batch = KVBatch(self.ctx, self.table, start, n_tokens=T, max_q=n) if n else None
            for li, kv in enumerate(self.kv if n else ()):
                k, v = (torch.randn(T, kv.n_kv, kv.head_dim, generator=g).to(torch.bfloat16).to(kv.device) for _ in range(2))
                kv_append(kv, batch, k, v)
                if self.keep_pages is not None:
                    kv_page_bounds(kv, batch, self.bounds[li])
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

    def _recount(self):
        """The host's lengths after replayed graphs of a harness over a pool: as they are on the device."""
        if self.pool is None:
            return
        if torch.cuda.is_current_stream_capturing():
            self.captured = True
        elif self.captured:
            self.lengths = self.ctx.tolist()
            self.pos = max(self.lengths)

    def _grow(self, seqs, n: int):
        """n more tokens of the sequences `seqs`, on the host's count."""
        if max(self.lengths[s] for s in seqs) + n > self.max_ctx:
            raise ValueError(f"{n} more tokens do not fit the cache's {self.max_ctx} positions")
        if self.pool is not None:
            pages = sum(-(-(m + n * (s in seqs)) // KV_PAGE) for s, m in enumerate(self.lengths)) - self.prefix * (self.n_seq - 1)
            if pages > self.pool.n_pages:
                raise ValueError(f"{n} more tokens need {pages} pages of a pool of {self.pool.n_pages}")
        for s in seqs:
            self.lengths[s] += n
        self.pos = max(self.lengths)

    def share_prefix(self, x: torch.Tensor) -> torch.Tensor:
        """A prompt that every sequence begins with, x fp32 [tokens][d]: through
        the layers once, as that of sequence 0; the others, which must be empty,
        begin with its whole pages, and a step reads these once for all (with
        keep_pages, those selected of them for each).  Returns
        what prefill returns; the prompt's tokens behind its last whole page are
        sequence 0's alone."""
        if self.cache == "dense" or self.pool is None:
            raise ValueError("share_prefix needs a pool of pages (n_pages)")
        self._recount()
        if any(self.lengths):
            raise ValueError("share_prefix needs empty sequences")
        y = self.prefill(x, 0)
        pages = x.shape[0] // KV_PAGE
        if pages and self.n_seq > 1:
            want = torch.full_like(self.ctx, pages * KV_PAGE)
            want[0] = x.shape[0]
            parent, shared = torch.zeros_like(want), torch.full_like(want, pages)
            parent[0] = -1
            kv_pages(self.pool, want, 0, parent=parent, shared=shared)
            self.lengths = [x.shape[0]] + [pages * KV_PAGE] * (self.n_seq - 1)
            self.prefix = pages
            self.shared.fill_(pages)
        return y

    def _attend(self, li: int, q: torch.Tensor, batch: KVBatch, workspace) -> torch.Tensor:
        kv = self.kv[li]
        if self.keep_pages is not None:
            kv_page_bounds(kv, batch, self.bounds[li])
        if batch is not self.one:
            return kv_attention(q, kv, batch, workspace=workspace)
        if self.keep_pages is not None:
            pages = kv_select(q, kv, batch, self.bounds[li], self.keep_pages, pages=self.picked, workspace=self.pick_ws)
            return kv_attention_selected(q, kv, batch, pages, workspace=workspace)
        if self.prefix:
            return kv_attention_shared(q, kv, batch, self.shared, workspace=self.share_ws)
        return kv_attention(q, kv, batch, workspace=workspace)

    def _paged(self, x: torch.Tensor, batch: KVBatch, workspace) -> torch.Tensor:
        """x fp32 [rows][d], the batch's rows, through every layer over the paged cache."""
        sh = self.shape
        H, KV, hd, d, T = sh.n_heads, sh.n_kv, sh.hd, sh.d, x.shape[0]
        for li, L in enumerate(self.layers):
            a = self._rmsnorm(x, self.g_attn[li])
            qkv = torch.nn.functional.linear(a, self.wqkv[li]).view(T, H + 2 * KV, hd)
            q, k, v = qkv.split([H, KV, KV], 1)
            q = kv_append(self.kv[li], batch, k, v, rot=self.rot_k, q=q, g_q=self.g_q[li], g_k=self.g_k[li], eps=EPS)
            att = self._attend(li, q, batch, workspace)
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
        self._recount()
        self._grow([seq], x.shape[0])
        out = []
        for p in x.split(MAX_PREFILL) if x.shape[0] else ():
            T = p.shape[0]
            if self.pool is None:
                self.ctx[seq:seq + 1].add_(T)
                start = torch.tensor([0, T], dtype=torch.int32, device=self.ctx.device)
                batch = KVBatch(self.ctx[seq:seq + 1], self.table[seq:seq + 1], start, n_tokens=T, max_q=T)
            else:
                want = self.ctx.clone()
                want[seq:seq + 1].add_(T)
                kv_pages(self.pool, want, T)
                # a prompt that was refused (only a captured one can be) has rows below position 0, which do not exist
                at = self.ctx * (self.ctx == want)
                start = torch.zeros_like(self.start)
                start[seq + 1:].fill_(T)
                batch = KVBatch(at, self.table, start, n_tokens=T, max_q=T)
            out.append(self._paged(p, batch, alloc_kv_workspace(self.kv[0], batch, self.shape.n_heads)))
        return torch.cat(out) if out else x

    def step(self, x: torch.Tensor) -> torch.Tensor:
        """x fp32 [n_seq][d] -> fp32 [n_seq][d] after every layer; the cache advances."""
        if self.cache != "dense":
            if x.shape != (self.n_seq, self.shape.d):
                raise ValueError("x must be [n_seq][d]")
            if self.pool is not None and torch.cuda.is_current_stream_capturing():
                self.captured = True
            self._grow(range(self.n_seq), 1)
            if self.pool is None:
                self.ctx.add_(1)
            else:
                torch.add(self.ctx, 1, out=self.want)
                kv_pages(self.pool, self.want, self.n_seq, q_start=self.start, slots=self.slots, status=self.status)
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
