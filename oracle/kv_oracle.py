"""CPU oracle of the paged 8-bit key/value cache -- TEST INFRASTRUCTURE ONLY.

Plain numpy.  Codes and scales are computed as the cache's definition has them
(norm and rotation in float64, one rounding to float32; scale = fp32(max|r| /
qmax); code = fp32(r / scale), clamped, rounded half-even), so they are
compared bit for bit; attention runs in float64.

``Cache`` holds the pages as ``include/prox.h`` lays them out:
  k [pages][n_kv][hp / 64][4][4][16][16]  indexes a b c d e: slot 16 b + d, channel 64 a + 16 c + e
  v [pages][n_kv][hp / 16][4][16][4][4]   indexes a b c d e: slot 16 d + 4 b + e, channel 16 a + c
"""

from __future__ import annotations

import numpy as np

PAGE = 64
QMAX = {"int8": 127.0, "fp8": 448.0}

_E4M3 = np.array([(1.0 + m / 8.0) * 2.0 ** (e - 7) if e else m / 8.0 * 2.0 ** -6
                  for e in range(16) for m in range(8)][:127])     # code 127 is NaN


def decode(kind: str, codes: np.ndarray) -> np.ndarray:
    """Codes (uint8) -> the numbers they stand for (float64)."""
    if kind == "int8":
        return codes.view(np.int8).astype(np.float64)
    mag = np.append(_E4M3, np.nan)[codes & 127]
    return np.where(codes & 128, -mag, mag)


def encode(kind: str, x: np.ndarray) -> np.ndarray:
    """Numbers in units of the scale -> codes (uint8): nearest, ties to even, clamped; NaN -> 0."""
    x = np.where(np.isnan(x), 0.0, np.asarray(x, dtype=np.float64))
    x = np.clip(x, -QMAX[kind], QMAX[kind])
    if kind == "int8":
        return np.rint(x).astype(np.int8).view(np.uint8)
    a = np.abs(x)
    hi = np.searchsorted(_E4M3, a).clip(0, 126)          # first code >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _E4M3[lo], _E4M3[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    code = np.where(up, hi, lo).astype(np.uint8)
    return np.where(np.signbit(x), code | 128, code).astype(np.uint8)


def head_pad(hd: int) -> int:
    return -(-hd // 64) * 64


class Cache:
    def __init__(self, kind: str, n_pages: int, n_kv: int, hd: int):
        self.kind, self.hd, self.hp, self.n_kv, self.n_pages = kind, hd, head_pad(hd), n_kv, n_pages
        self.k = np.zeros((n_pages, n_kv, PAGE * self.hp), np.uint8)
        self.v = np.zeros_like(self.k)
        self.ks = np.zeros((n_pages, n_kv), np.float32)
        self.vs = np.zeros_like(self.ks)

    def tokens(self, which: str) -> np.ndarray:
        """Codes as [pages][n_kv][slot][channel] (a copy)."""
        P, K, hp = self.n_pages, self.n_kv, self.hp
        if which == "k":
            x = self.k.reshape(P, K, hp // 64, 4, 4, 16, 16).transpose(0, 1, 3, 5, 2, 4, 6)
        else:
            x = self.v.reshape(P, K, hp // 16, 4, 16, 4, 4).transpose(0, 1, 5, 3, 6, 2, 4)
        return np.ascontiguousarray(x).reshape(P, K, PAGE, hp)

    def put(self, which: str, tok: np.ndarray) -> None:
        P, K, hp = self.n_pages, self.n_kv, self.hp
        if which == "k":
            x = tok.reshape(P, K, 4, 16, hp // 64, 4, 16).transpose(0, 1, 4, 2, 5, 3, 6)
            self.k = np.ascontiguousarray(x).reshape(P, K, PAGE * hp)
        else:
            x = tok.reshape(P, K, 4, 4, 4, hp // 16, 16).transpose(0, 1, 5, 3, 6, 2, 4)
            self.v = np.ascontiguousarray(x).reshape(P, K, PAGE * hp)


def rows_of(q_start, ctx, n_tokens, max_q):
    """(sequence, row, position) of every row that a call works on."""
    out = []
    for s in range(len(ctx)):
        q0, q1 = (s, s + 1) if q_start is None else (int(q_start[s]), int(q_start[s + 1]))
        for i in range(min(q1 - q0, max_q)):
            out.append((s, q0 + i, int(ctx[s]) - (q1 - q0) + i))
    return out


def turn(x, pos, rot, pairing, gain, eps):
    """Norm (gain given) and rotation (rot [rows][rd / 2][2] given) of heads x
    [heads][hd] at position pos, float64."""
    x = np.asarray(x, dtype=np.float64)
    if gain is not None:
        x = x / np.sqrt(np.mean(x * x, axis=-1, keepdims=True) + np.float64(np.float32(eps))) * np.asarray(gain, dtype=np.float64)
    if rot is None:
        return x
    c, s = rot[pos, :, 0].astype(np.float64), rot[pos, :, 1].astype(np.float64)
    h = c.size
    y = x.copy()
    ia, ib = (np.arange(h), np.arange(h) + h) if pairing == "halves" else (2 * np.arange(h), 2 * np.arange(h) + 1)
    a, b = x[..., ia], x[..., ib]
    y[..., ia], y[..., ib] = a * c - b * s, a * s + b * c
    return y


def append(cache: Cache, table, ctx, q_start, max_q, k, v, rot=None, pairing="interleaved", g_k=None, eps=1e-5):
    """k, v float64 [n_tokens][n_kv][hd] (values of the bf16 inputs)."""
    f32 = np.float32
    todo = {}
    for s, row, pos in rows_of(q_start, ctx, len(k), max_q):
        if 0 <= pos < PAGE * table.shape[1] and 0 <= table[s, pos // PAGE] < cache.n_pages:
            todo.setdefault((s, pos // PAGE), []).append((row, pos))
    kt, vt = cache.tokens("k"), cache.tokens("v")
    for (s, pg), items in todo.items():
        page = int(table[s, pg])
        slots = [p % PAGE for _, p in items]
        for tok, sc, new in ((kt, cache.ks, np.stack([turn(k[r], p, rot, pairing, g_k, eps) for r, p in items])),
                             (vt, cache.vs, np.stack([v[r] for r, _ in items]))):
            with np.errstate(over="ignore", invalid="ignore"):
                r = new.astype(f32)                                       # [n][n_kv][hd]
            for h in range(cache.n_kv):
                fresh = slots[0] == 0
                old = f32(0) if fresh else sc[page, h]
                fin = np.abs(r[:, h][np.isfinite(r[:, h])])
                most = f32(fin.max()) if fin.size else f32(0)
                now = max(old, f32(most / f32(QMAX[cache.kind])))
                if fresh:
                    tok[page, h] = 0
                elif now > old > 0:
                    val = (decode(cache.kind, tok[page, h]).astype(f32) * old).astype(f32)
                    tok[page, h] = encode(cache.kind, (val / now).astype(f32))
                if now > 0:
                    with np.errstate(invalid="ignore"):
                        tok[page, h, slots, :cache.hd] = encode(cache.kind, (r[:, h] / now).astype(f32))
                else:
                    tok[page, h, slots, :cache.hd] = 0
                sc[page, h] = now
    cache.put("k", kt)
    cache.put("v", vt)


def gather(cache: Cache, table, s, lo, hi):
    """Values of positions lo .. hi - 1 of sequence s (float64 [n][n_kv][hd], k
    and v) and whether their page exists."""
    pos = np.arange(lo, hi)
    page = table[s, pos // PAGE]
    there = (page >= 0) & (page < cache.n_pages)
    page = np.where(there, page, 0)
    out = []
    for codes, sc, which in ((cache.k, cache.ks, "k"), (cache.v, cache.vs, "v")):
        d, j = np.arange(cache.hd)[None, :], (pos % PAGE)[:, None]
        if which == "k":
            at = (((d // 64 * 4 + j // 16) * 4 + d % 64 // 16) * 16 + j % 16) * 16 + d % 16
        else:
            at = (((d // 16 * 4 + j % 16 // 4) * 16 + d % 16) * 4 + j // 16) * 4 + j % 4
        c = codes[page[:, None], :, at]                                     # [n][hd][n_kv]
        out.append(decode(cache.kind, np.ascontiguousarray(c)).transpose(0, 2, 1) * sc[page].astype(np.float64)[:, :, None])
    return out[0], out[1], there


def attention(cache: Cache, table, ctx, q_start, max_q, q, scale, window=0, n_out=None):
    """q float64 [n_tokens][H][hd].  Returns (out, tol): float64 results (NaN on
    rows that no sequence has) and a bound of the kernel's error at each.

    Weights p_j are rounded to fp16: relative error at most u = 2^-11, or 2^-33
    of the largest weight where they are fp16 subnormals (they are held 2^8
    larger).  The result is the mean with the rounded weights' own sum below it,
    so relative errors e_j of the weights move it by sum_j w_j e_j (v_j - o) to
    first order.  e_j also holds the score's error (of the exponent, absolute):
      - fp32 sums of hd products: for e4m3 at most hd + 8 roundings of 2^-24 of
        scale sum_d |q_d k_d|; for int8, whose codes are taken as 1024 + 128 + c
        with -1152 sum(q) as start, hd / 2 roundings (a matrix instruction adds
        32 products with no more than 8) of sums up to (1152 + 1279) sum(|q|)
        units of the key's scale;
      - q's channels below 2^-17 of the row's largest are off by 2^-25 of that;
    and 2^-21 for exp2.  The sums over the keys: a page adds two matrix
    instructions' 32 products to the running sums, with no more than 8 roundings
    each, and takes part in at most one rescaling and one join of parts (3
    roundings), all of sums up to sum_j w_j |v_j|: 20 a page, and 20 for the rest.
    The bf16 result is rounded by at most 2^-8 |o|.  A weight under 2^-126 of the
    row's largest is no normal fp32 number and may be taken as 0.  All channels
    of a row share a unit: where its largest sum is 2^99 units and more (weights
    held 2^10 large at most, so 2^89 over sum_j p_j <= n in the mean), a page of
    values too small for that unit counts as a quarter of it at most, codes up
    to 448: an error of 2^7 against n^-1 2^89, n 2^-82 of the largest of
    sum_j w_j |v_j| over the channels."""
    T, H, hd = q.shape
    out = np.full((T, H, hd), np.nan)
    tol = np.zeros((T, H, hd))
    rep = H // cache.n_kv
    u, r24, big = 2.0 ** -11, 2.0 ** -24, 1152 + 1279
    int8 = cache.kind == "int8"
    vals = {}
    for s, row, pos in rows_of(q_start, ctx, T, max_q):
        if pos < 0 or pos >= PAGE * table.shape[1]:
            out[row] = 0
            continue
        if s not in vals:
            last = min(int(ctx[s]), PAGE * table.shape[1])
            got = gather(cache, table, s, 0, max(last, 1))
            page = np.where(got[2], table[s, np.arange(max(last, 1)) // PAGE], 0)
            vals[s] = got + (cache.ks[page].astype(np.float64),)
        K, V, there, KS = vals[s]
        lo = max(0, pos - window + 1) if window else 0
        see = np.flatnonzero(there[lo:pos + 1]) + lo
        if see.size == 0:
            out[row] = 0
            continue
        for h in range(H):
            k, v = K[see, h // rep], V[see, h // rep]
            z = k @ q[row, h] * scale
            w = np.exp(z - z.max())
            w /= w.sum()
            o = w @ v
            aq = np.abs(q[row, h])
            unit_k = KS[see, h // rep]
            if int8:
                eta = hd / 2 * r24 * big * unit_k * aq.sum() + 8 * r24 * (np.abs(k) @ aq)
            else:
                eta = (hd + 8) * r24 * (np.abs(k) @ aq)
            eta = abs(scale) * (eta + 2.0 ** -25 * aq.max() * np.abs(k).sum(-1)) + 2.0 ** -21
            pages = see.size / PAGE + 2
            sums = 20 * (pages + 1) * r24 * (w @ np.abs(v))
            out[row, h] = o
            tol[row, h] = (2.0 ** -8 * np.abs(o) + (w * (1.02 * (u + eta))) @ np.abs(v - o) + sums
                           + see.size * 2.0 ** -33 * np.abs(v - o).max(0) + 1e-37
                           + see.size * 2.0 ** -82 * (w @ np.abs(v)).max())
    return out, tol
