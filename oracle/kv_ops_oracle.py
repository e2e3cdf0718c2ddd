"""CPU oracle of the operators around the paged 8-bit cache -- TEST INFRASTRUCTURE ONLY.

Plain numpy, one sequence, page and row at a time, from the definitions in
``include/prox.h``: page tables (whole numbers), bounds of keys (whole numbers),
selection of pages (whole numbers and two fp32 roundings), and the attentions
over selected pages and with a shared prefix as ``kv_oracle.attention`` over what
each row sees.
"""

from __future__ import annotations

import numpy as np

from oracle import kv_oracle as KO

PAGE = 64


class Pool:
    def __init__(self, n_pages, n_seq, max_pages):
        self.refs = np.zeros(n_pages, np.int32)
        self.ctx = np.zeros(n_seq, np.int32)
        self.table = np.full((n_seq, max_pages), -1, np.int32)

    def move(self, want, n_rows, parent=None, shared=None):
        """(q_start, slots, status) of a call; the pool follows."""
        n, width = self.table.shape
        start, had = self.ctx.copy(), self.ctx.copy()
        want = [max(int(w), 0) for w in want]
        if parent is not None:
            for s in range(n):
                p = int(parent[s])
                if had[s] == 0 and 0 <= p < n:
                    first = max(min(int(shared[s]), int(had[p]) // PAGE), 0)
                    for j in range(first):
                        self.table[s, j] = self.table[p, j]
                        self.refs[self.table[p, j]] += 1
                    start[s] = PAGE * first
        for s in range(n):
            for j in range(-(-want[s] // PAGE), -(-int(start[s]) // PAGE)):
                self.refs[self.table[s, j]] -= 1
                self.table[s, j] = -1
        free = [p for p in range(len(self.refs)) if self.refs[p] == 0]
        held = self.refs.copy()
        refused, asked, taken = 0, 0, 0
        q_start, slots = [0], np.full(n_rows, -1, np.int32)
        for s in range(n):
            has, needs = -(-int(start[s]) // PAGE), -(-want[s] // PAGE)
            no = needs > width
            if want[s] > start[s] and start[s] % PAGE:
                no = no or held[self.table[s, start[s] // PAGE]] > 1
            more = 0 if no else max(needs - has, 0)
            asked += more
            no = no or (more > 0 and asked > len(free))
            length = int(start[s]) if no else want[s]
            refused += no
            if not no:
                for j in range(has, needs):
                    self.table[s, j] = free[asked - more + j - has]
                    self.refs[self.table[s, j]] = 1
                    taken = asked
            for pos in range(int(start[s]), length):
                row = q_start[-1] + pos - int(start[s])
                if row < n_rows:
                    slots[row] = PAGE * self.table[s, pos // PAGE] + pos % PAGE
            q_start.append(q_start[-1] + max(length - int(start[s]), 0))
            self.ctx[s] = length
        return np.array(q_start, np.int32), slots, np.array([refused, len(free) - taken], np.int32)


def bounds(cache, table, ctx, q_start, n_tokens, max_q, out):
    """Set the bounds of the pages that the batch's tokens lie in."""
    tok = cache.tokens("k")
    seen = {}
    for s, _, pos in KO.rows_of(q_start, ctx, n_tokens, max_q):
        if 0 <= pos < PAGE * table.shape[1] and 0 <= table[s, pos // PAGE] < cache.n_pages:
            seen[s, pos // PAGE] = max(seen.get((s, pos // PAGE), 0), pos % PAGE + 1)
    for (s, pg), held in seen.items():
        page = int(table[s, pg])
        v = KO.decode(cache.kind, tok[page, :, :held])                     # [n_kv][held][hp]
        v = np.where(np.isnan(v), 0.0, v)
        lo, hi = v.min(1), v.max(1)
        if cache.kind == "fp8":
            lo, hi = np.floor(lo * 127 / 448), np.ceil(hi * 127 / 448)
        out[page, :, 0], out[page, :, 1] = lo, hi


def select(cache, table, ctx, q_start, max_q, q, bnd, keep, first, last, out):
    """q float64 [n_tokens][H][hd] (values of the bf16 inputs); rows of the batch are set in out."""
    f32 = np.float32
    T, H, hd = q.shape
    rep = H // cache.n_kv
    for s, row, pos in KO.rows_of(q_start, ctx, T, max_q):
        out[row] = -1
        if not 0 <= pos < PAGE * table.shape[1]:
            continue
        n = pos // PAGE + 1
        x = q[row].astype(f32)
        fin = np.where(np.isfinite(x), np.abs(x), f32(0))
        unit = (fin.max(-1) / f32(127)).astype(f32)                        # [H]
        with np.errstate(invalid="ignore", over="ignore"):
            r = (x / np.where(unit > 0, unit, f32(1))[:, None]).astype(f32)
            q8 = np.rint(np.clip(np.where(np.isnan(r), f32(0), r), -127, 127)).astype(np.int64)
        for g in range(cache.n_kv):
            keys = []
            for p in range(n):
                page = int(table[s, p])
                if not 0 <= page < cache.n_pages:
                    continue
                lo, hi = (bnd[page, g, i, :hd].astype(np.int64) for i in (0, 1))
                a = q8[g * rep:(g + 1) * rep]
                dot = (np.minimum(a, 0) * lo + np.maximum(a, 0) * hi).sum(-1)   # sum max(a lo, a hi) where lo <= hi
                with np.errstate(invalid="ignore", over="ignore"):
                    t = (dot.astype(f32) * unit[g * rep:(g + 1) * rep]).astype(f32).max()
                    key = f32(t * cache.ks[page, g])
                key = (0, -np.inf) if np.isnan(key) else (1, float(key))
                if p < first or p >= n - last:
                    key = (2, 0.0)
                keys.append((-key[0], -key[1], p))
            kept = sorted(p for _, _, p in sorted(keys)[:keep])
            out[row, g, :len(kept)] = kept


class _Part:
    """The pages of a cache's one key head, in the order of a list (for kv_oracle.attention)."""

    def __init__(self, cache, head):
        self.kind, self.hd, self.hp, self.n_kv, self.n_pages = cache.kind, cache.hd, cache.hp, 1, cache.n_pages
        self.k, self.v = cache.k[:, head:head + 1], cache.v[:, head:head + 1]
        self.ks, self.vs = cache.ks[:, head:head + 1], cache.vs[:, head:head + 1]


def attention_selected(cache, table, ctx, q_start, max_q, q, pages, scale):
    """(out, tol) as kv_oracle.attention, of rows that see the listed pages alone: a
    list ends before the first entry that is not above the one before it, or is
    behind the row's own page."""
    T, H, hd = q.shape
    rep = H // cache.n_kv
    out, tol = np.full((T, H, hd), np.nan), np.zeros((T, H, hd))
    for s, row, pos in KO.rows_of(q_start, ctx, T, max_q):
        for g in range(cache.n_kv):
            heads = slice(g * rep, (g + 1) * rep)
            ok = []
            for p in pages[row, g] if 0 <= pos < PAGE * table.shape[1] else ():
                if not (ok[-1] if ok else -1) < p <= pos // PAGE:
                    break
                ok.append(int(p))
            if not ok:
                out[row, heads] = 0
                continue
            # a sequence of the listed pages: whole ones, and the row's own last
            t = table[s, ok][None]
            n = PAGE * len(ok) if ok[-1] < pos // PAGE else PAGE * (len(ok) - 1) + pos % PAGE + 1
            o, e = KO.attention(_Part(cache, g), t, np.array([n]), np.array([0, 1]), 1, q[row:row + 1, heads], scale)
            out[row, heads], tol[row, heads] = o[0], e[0]
    return out, tol


def attention_shared(cache, table, ctx, q_start, max_q, q, shared, group_start, scale):
    """(out, tol) as kv_oracle.attention, with the first pages of a group's sequences taken
    from its first one."""
    table = table.copy()
    n, width = table.shape
    q0 = np.arange(n + 1) if q_start is None else np.asarray(q_start)
    gs = [0, n] if group_start is None else [int(x) for x in group_start]
    own = table.copy()
    for g, (a, b) in enumerate(zip(gs, gs[1:])):
        pages = min(max(int(shared[g]), 0), width)
        for s in range(a, b):
            if int(ctx[s]) - int(q0[s + 1] - q0[s]) >= PAGE * pages:
                table[s, :pages] = own[a, :pages]
    return KO.attention(cache, table, ctx, q_start, max_q, q, scale)
