"""GPU checks of the paged 8-bit key/value cache against oracle/kv_oracle.py.

Append and read: codes, scales, rotated queries and read values bit for bit
(norm and rotation run in float64 on both sides).  Attention: the bound that
``kv_oracle.attention`` derives for every element from the roundings made."""

import numpy as np
import pytest
import torch

from oracle import kv_oracle as KO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bf16(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16)


def f64(t):
    return t.detach().double().cpu().numpy()


def rope_table(rows, rot_dim, theta=10000.0):
    i = torch.arange(rot_dim // 2, dtype=torch.float64)
    ang = torch.arange(rows, dtype=torch.float64)[:, None] * (theta ** (-2.0 * i / rot_dim))[None]
    return torch.view_as_real(torch.polar(torch.ones_like(ang), ang)).float().contiguous()


class World:
    """A cache with its pages in random order and stale bytes in them, on the
    GPU and in the oracle, and the sequences' table."""

    def __init__(self, kind, H, KV, hd, caps, seed=0, extra=2):
        import free_ffn_activation_prox_amd as P
        self.P, self.kind, self.H, self.KV, self.hd = P, kind, H, KV, hd
        self.rng = np.random.default_rng(seed)
        need = [-(-c // 64) for c in caps]
        n_pages = sum(need) + extra
        order = self.rng.permutation(n_pages).astype(np.int32)
        self.table = np.full((len(caps), max(need)), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.table[s, :n] = order[at:at + n]
            at += n
        self.o = KO.Cache(kind, n_pages, KV, hd)
        self.o.k = self.rng.integers(0, 256, self.o.k.shape).astype(np.uint8)
        self.o.v = self.rng.integers(0, 256, self.o.v.shape).astype(np.uint8)
        self.o.ks = self.rng.random(self.o.ks.shape).astype(np.float32)
        self.o.vs = self.rng.random(self.o.vs.shape).astype(np.float32)
        self.c = P.KVCache(kind, hd, *(torch.from_numpy(a.copy()).cuda() for a in (self.o.k, self.o.v, self.o.ks, self.o.vs)))
        self.ctx = np.zeros(len(caps), np.int32)
        self.rot = rope_table(64 * self.table.shape[1], hd if hd % 16 == 0 else hd // 16 * 16 or 2)

    def batch(self, new, advance=True, pad=0, max_q=None):
        """Batch of the next new[s] tokens of every sequence (pad rows behind the last)."""
        if advance:
            self.ctx = self.ctx + np.asarray(new, np.int32)
        start = np.concatenate([[0], np.cumsum(new)]).astype(np.int32)
        b = self.P.KVBatch(torch.from_numpy(self.ctx.copy()).cuda(), torch.from_numpy(self.table).cuda(),
                           torch.from_numpy(start).cuda(), n_tokens=int(start[-1]) + pad,
                           max_q=int(max(new)) if max_q is None else max_q)
        return b, start

    def rows(self, n, heads, scale=1.0):
        return bf16(self.rng.standard_normal((n, heads, self.hd)) * scale).cuda()

    def append(self, new, *, pairing="interleaved", norm=False, rotate=True, pad=0, grow=1.0, packed=False, inplace=False):
        P, hd = self.P, self.hd
        b, start = self.batch(new, pad=pad)
        T = b.n_tokens
        if packed:
            x = bf16(self.rng.standard_normal((T, (self.H + 2 * self.KV) * hd + 8)) * grow).cuda()
            q, k, v, _ = x.split([self.H * hd, self.KV * hd, self.KV * hd, 8], 1)
            q, k, v = q.view(T, self.H, hd), k.view(T, self.KV, hd), v.view(T, self.KV, hd)
        else:
            q, k, v = self.rows(T, self.H, grow), self.rows(T, self.KV, grow), self.rows(T, self.KV, grow)
        g_q = g_k = None
        if norm:
            g_q, g_k = (torch.from_numpy((1 + 0.1 * self.rng.standard_normal(hd)).astype(np.float32)).cuda() for _ in range(2))
        rot = self.rot if rotate else None
        qh, kh, vh = f64(q), f64(k), f64(v)
        out = q if inplace else torch.full((T, self.H, hd), 7.0, dtype=torch.bfloat16, device="cuda")
        got = P.kv_append(self.c, b, k, v, rot=None if rot is None else rot.cuda(), q=q, q_out=out, g_q=g_q, g_k=g_k,
                          pairing=pairing)
        torch.cuda.synchronize()
        assert got is out
        rn = None if rot is None else rot.numpy()
        KO.append(self.o, self.table, self.ctx, start, b.max_q, kh, vh, rn, pairing, None if g_k is None else f64(g_k))
        want = qh.copy() if inplace else np.full((T, self.H, hd), 7.0)
        for s, row, pos in KO.rows_of(start, self.ctx, T, b.max_q):
            if 0 <= pos < 64 * self.table.shape[1]:
                want[row] = f64(bf16(KO.turn(qh[row], pos, rn, pairing, None if g_q is None else f64(g_q), 1e-5)))
            else:
                want[row] = 0
        assert np.array_equal(f64(got), want), "queries differ"
        self.same_cache()
        return b, start, got

    def same_cache(self):
        for n, a, b in (("k scale", self.c.k_scale, self.o.ks), ("v scale", self.c.v_scale, self.o.vs),
                        ("k codes", self.c.k, self.o.k), ("v codes", self.c.v, self.o.v)):
            assert np.array_equal(a.cpu().numpy(), b), f"{n} differ"

    def attend(self, b, start, q=None, window=0, scale=None, **kw):
        q = self.rows(b.n_tokens, self.H, 1.5) if q is None else q
        out = torch.full(q.shape, 7.0, dtype=torch.bfloat16, device="cuda")
        self.P.kv_attention(q, self.c, b, out=out, window=window, scale=scale, **kw)
        torch.cuda.synchronize()
        want, tol = KO.attention(self.o, self.table, self.ctx, start, b.max_q, f64(q),
                                 self.hd ** -0.5 if scale is None else scale, window)
        got = f64(out)
        idle = np.isnan(want).all((1, 2))
        assert np.array_equal(got[idle], np.full_like(got[idle], 7.0)), "rows outside the sequences were written"
        err = np.abs(got[~idle] - want[~idle])
        worst = float(np.max(err / tol[~idle].clip(1e-37))) if err.size else 0.0
        assert np.isfinite(got[~idle]).all() and worst <= 1.0, f"error {worst:.3f} of the bound"
        return out, worst


def settle(w, new):
    """Fill the cache of a world: `new` tokens of every sequence, in one call."""
    w.append(new, rotate=False)


CASES = [
    # kind, H, KV, hd, pairing, norm
    ("int8", 4, 2, 64, "interleaved", False),
    ("fp8", 6, 6, 128, "halves", True),
    ("int8", 7, 1, 80, "halves", True),
    ("fp8", 2, 2, 96, "interleaved", True),
    ("int8", 3, 3, 8, "interleaved", True),
    ("fp8", 5, 1, 16, "halves", False),
    ("int8", 2, 1, 256, "halves", False),
    ("fp8", 4, 2, 192, "interleaved", False),
]


@pytest.mark.parametrize("kind,H,KV,hd,pairing,norm", CASES)
def test_append_bit_exact_over_several_calls(kind, H, KV, hd, pairing, norm):
    w = World(kind, H, KV, hd, [200, 64, 1, 130], seed=hd)
    # begins inside and at the edges of pages, empty sequences, one token, growing scales, rows behind the last
    w.append([1, 0, 0, 60], pairing=pairing, norm=norm)
    w.append([1, 64, 1, 4], pairing=pairing, norm=norm, grow=2.0, packed=True, pad=3)
    w.append([125, 0, 0, 1], pairing=pairing, norm=norm, grow=0.5, inplace=True)
    w.append([1, 0, 0, 65], pairing=pairing, norm=norm, grow=3.0)
    w.append([70, 0, 0, 0], pairing=pairing, norm=norm, packed=True)


def test_append_without_rotation_queries_or_norm_of_one_side():
    w = World("int8", 2, 2, 64, [70], seed=3)
    w.append([70], rotate=False)
    P = w.P
    b, start = w.batch([1], advance=False)
    k, v = w.rows(1, 2, 5.0), w.rows(1, 2, 5.0)
    assert P.kv_append(w.c, b, k, v) is None
    KO.append(w.o, w.table, w.ctx, start, 1, f64(k), f64(v))
    w.same_cache()


def test_append_positions_and_pages_that_do_not_exist():
    for kind in ("int8", "fp8"):
        w = World(kind, 2, 1, 64, [192, 192, 192], seed=5)
        w.table[1, 1] = w.o.n_pages          # one past the last page
        w.table[2, 0] = -5
        w.ctx[:] = [150, 20, 0]              # sequence 0 runs over its 192 positions
        w.append([70, 130, 100])
        w.ctx[:] = [-40, 5, 0]               # rows before position 0
        w.append([30, 20, 3])


def test_append_max_q_bounds_the_rows():
    w = World("int8", 2, 1, 64, [300], seed=6)
    P = w.P
    b, start = w.batch([200], max_q=70)
    k, v, q = w.rows(200, 1), w.rows(200, 1), w.rows(200, 2)
    out = torch.full_like(q, 7.0)
    P.kv_append(w.c, b, k, v, q=q, q_out=out)
    KO.append(w.o, w.table, w.ctx, start, 70, f64(k), f64(v))
    w.same_cache()
    assert torch.equal(out[:70], q[:70]) and bool((out[70:] == 7).all())


def test_append_infinities_nan_zeros_and_tiny_values():
    for kind in ("int8", "fp8"):
        w = World(kind, 1, 2, 64, [64, 64, 64], seed=7)
        P = w.P
        b, start = w.batch([5, 4, 3])
        k, v = w.rows(12, 2), w.rows(12, 2)
        k[1, 0, 3], k[2, 1, 5], v[0, 1, 7] = float("inf"), float("nan"), float("-inf")
        k[5:9] = 0                            # a page of zeros
        v[5:9] = float("inf")                 # and one without a finite value
        k[9:] *= 2.0 ** -118                  # scales below the normal numbers
        v[9:] *= 1e36
        P.kv_append(w.c, b, k, v)
        with np.errstate(all="ignore"):
            KO.append(w.o, w.table, w.ctx, start, b.max_q, f64(k), f64(v))
        w.same_cache()


@pytest.mark.parametrize("kind,H,KV,hd", [("int8", 2, 2, 64), ("fp8", 3, 3, 80), ("int8", 1, 1, 8), ("fp8", 1, 1, 256)])
def test_read_bit_exact(kind, H, KV, hd):
    w = World(kind, H, KV, hd, [200, 64, 10], seed=hd + 1)
    settle(w, [190, 64, 10])
    w.table[0, 1] = -1                        # a page that is not there reads as zeros
    w.ctx[2] = 4                              # rows before position 0 read as zeros
    b, start = w.batch([190, 1, 10], advance=False, pad=2)
    for dt in (torch.float32, torch.bfloat16):
        ko, vo = (torch.full((b.n_tokens, KV, hd), 7.0, dtype=dt, device="cuda") for _ in range(2))
        w.P.kv_read(w.c, b, dtype=dt, k_out=ko, v_out=vo)
        kw, vw = (np.full((b.n_tokens, KV, hd), 7.0) for _ in range(2))
        for s, row, pos in KO.rows_of(start, w.ctx, b.n_tokens, b.max_q):
            kw[row] = vw[row] = 0
            if pos >= 0:
                k, v, there = KO.gather(w.o, w.table, s, pos, pos + 1)
                if there[0]:
                    kw[row], vw[row] = k[0].astype(np.float32), v[0].astype(np.float32)
        if dt == torch.bfloat16:
            kw, vw = f64(bf16(kw)), f64(bf16(vw))
        assert np.array_equal(f64(ko), kw) and np.array_equal(f64(vo), vw)


# one token a sequence: lengths around pages, long ones, many heads of a group
@pytest.mark.parametrize("kind,H,KV,hd", [("int8", 4, 4, 64), ("fp8", 8, 2, 128), ("int8", 7, 1, 128), ("fp8", 20, 1, 80),
                                          ("int8", 34, 2, 96), ("int8", 4, 2, 256), ("fp8", 2, 1, 192), ("int8", 3, 3, 8)])
def test_attention_single_tokens(kind, H, KV, hd):
    lens = [1, 2, 15, 16, 17, 63, 64, 65, 128, 129, 700, 1500]
    w = World(kind, H, KV, hd, lens, seed=H * hd)
    settle(w, lens)
    b, start = w.batch([1] * len(lens), advance=False)
    worst = w.attend(b, start)[1]
    print(f"[kv] single tokens {kind} H={H} KV={KV} hd={hd}: {worst:.3f} of the bound", flush=True)
    for window in (1, 2, 64, 100, 5000):
        w.attend(b, start, window=window)
    # without q_start
    one = w.P.KVBatch(b.ctx_len, b.block_table)
    w.attend(one, None)


@pytest.mark.parametrize("kind,H,KV,hd", [("int8", 2, 2, 64), ("fp8", 4, 1, 128), ("int8", 5, 1, 96), ("fp8", 3, 1, 256),
                                          ("int8", 16, 2, 128), ("int8", 2, 1, 192)])
def test_attention_prompts_and_chunks(kind, H, KV, hd):
    lens = [300, 64, 65, 1, 90, 1000]
    w = World(kind, H, KV, hd, lens, seed=H + hd)
    settle(w, lens)
    for new in ([300, 64, 65, 1, 90, 1], [3, 1, 2, 1, 0, 5], [0, 0, 33, 0, 0, 700], [1, 1, 1, 1, 1, 200]):
        b, start = w.batch(new, advance=False, pad=2)
        worst = w.attend(b, start)[1]
        print(f"[kv] {new} {kind} H={H} KV={KV} hd={hd}: {worst:.3f} of the bound", flush=True)
        w.attend(b, start, window=50)
        w.attend(b, start, window=1)


def test_attention_long_single_sequence():
    for kind, n in (("int8", 20000), ("fp8", 9001)):
        w = World(kind, 8, 1, 128, [n], seed=n)
        settle(w, [n])
        for new in ([1], [3], [70]):
            b, start = w.batch(new, advance=False)
            w.attend(b, start)
            w.attend(b, start, window=4096)


def test_attention_missing_pages_and_rows_without_keys():
    w = World("int8", 4, 2, 64, [400, 300, 200, 64], seed=11)
    settle(w, [400, 300, 200, 64])
    w.table[0, 2:4] = -1                      # a hole
    w.table[1, :] = w.o.n_pages               # no page at all: zeros
    w.table[2, 0] = 1 << 30
    w.ctx[3] = 2                              # four rows, two of them before position 0
    for new in ([1, 1, 1, 4], [350, 20, 200, 4]):
        b, start = w.batch(new, advance=False)
        out, _ = w.attend(b, start)
        assert not out[start[1]:start[2]].any() and not out[start[3]:start[3] + 2].any()
        w.attend(b, start, window=70)
    w.ctx[:] = [64 * 7 + 3, 0, -7, 1 << 30]   # past the table, empty, negative, far past
    b, start = w.batch([5, 1, 1, 1], advance=False)
    w.attend(b, start)


def test_attention_unwritten_slots_and_spread_values():
    # stale bytes (NaN codes among them) behind the last token; scores of +-hundreds; pages of unlike scale
    for kind in ("int8", "fp8"):
        w = World(kind, 4, 1, 64, [400, 64, 130], seed=13)
        for part, grow in (([30, 1, 70], 1.0), ([100, 0, 58], 300.0), ([200, 0, 1], 0.01), ([37, 0, 0], 30.0)):
            w.append(part, grow=grow, rotate=False)
        w.o.k, w.o.v = (c.copy() for c in (w.o.k, w.o.v))
        for s in range(3):                    # every slot behind the last token: all ones, a NaN code
            p, n = int(w.table[s, w.ctx[s] // 64]) if w.ctx[s] % 64 else -1, int(w.ctx[s] % 64)
            if p >= 0:
                for which in ("k", "v"):
                    t = w.o.tokens(which)
                    t[p, :, n:] = 0xff
                    w.o.put(which, t)
        w.c.k.copy_(torch.from_numpy(w.o.k))
        w.c.v.copy_(torch.from_numpy(w.o.v))
        for new in ([1, 1, 1], [300, 1, 129]):
            b, start = w.batch(new, advance=False)
            for scale in (None, 3.0, 0.0, -0.1, 1e-30):
                w.attend(b, start, scale=scale)


def test_attention_many_tiny_weights_beside_a_large_one():
    # one key with weight 1 and value 0, thousands of weight 2^-24 each: their
    # sum, 2^-12, is the whole result
    for kind in ("int8", "fp8"):
        n, hd = 4097, 64
        w = World(kind, 2, 1, hd, [n], seed=41)
        k, v = torch.zeros(n, 1, hd, dtype=torch.bfloat16), w.rows(n, 1).cpu().abs() + 1
        k[0, 0, 0] = 1.0
        v[0] = 0
        b, start = w.batch([n])
        w.P.kv_append(w.c, b, k.cuda(), v.cuda())
        KO.append(w.o, w.table, w.ctx, start, n, f64(k), f64(v))
        w.same_cache()
        q = torch.zeros(n, 2, hd, dtype=torch.bfloat16, device="cuda")
        q[:, :, 0] = 1.0
        for new in (1, 100):
            b, start = w.batch([new], advance=False)
            out, _ = w.attend(b, start, q=q[:new].clone(), scale=24.0 * float(np.log(2.0)))
            assert float(out[-1].float().abs().min()) > 2e-4


def test_attention_bad_query_stays_in_its_row():
    w = World("int8", 4, 1, 128, [200], seed=17)
    settle(w, [200])
    for n in (2, 40):
        b, start = w.batch([n], advance=False)
        q = w.rows(n, 4)
        good, _ = w.attend(b, start, q=q.clone())
        bad = q.clone()
        bad[1, 2, 5] = float("nan")
        out = w.P.kv_attention(bad, w.c, b)
        keep = torch.ones(n, 4, dtype=torch.bool)
        keep[1, 2] = False
        assert torch.equal(out.cpu()[keep], good.cpu()[keep]) and bool(out[1, 2].isnan().all())


def test_attention_strides_and_stale_workspace():
    w = World("fp8", 8, 2, 128, [700, 90], seed=19)
    settle(w, [700, 90])
    for new in ([1, 1], [260, 90]):
        b, start = w.batch(new, advance=False)
        T = b.n_tokens
        q = w.rows(T, 8)
        ref, _ = w.attend(b, start, q=q)
        wide = torch.zeros(T, 8 * 128 + 264, dtype=torch.bfloat16, device="cuda")
        qs = wide[:, 8:8 + 8 * 128].view(T, 8, 128)
        qs.copy_(q)
        into = torch.full((T, 8 * 128 + 64), 7.0, dtype=torch.bfloat16, device="cuda")
        os_ = into[:, 64:].view(T, 8, 128)
        ws = w.P.alloc_kv_workspace(w.c, b, 8)
        for fill in (0, 0xff):
            ws.fill_(fill)
            w.P.kv_attention(qs, w.c, b, out=os_, workspace=ws)
            assert torch.equal(os_, ref) and bool((into[:, :64] == 7).all())


def test_python_refusals_on_the_gpu():
    w = World("int8", 4, 2, 64, [64], seed=23)
    P = w.P
    b, _ = w.batch([4])
    q, k, v = w.rows(4, 4), w.rows(4, 2), w.rows(4, 2)
    for call in (lambda: P.kv_append(w.c, b, k.float(), v), lambda: P.kv_append(w.c, b, k[:, :1], v),
                 lambda: P.kv_append(w.c, b, k, v[:3]), lambda: P.kv_append(w.c, b, k, v, pairing="thirds"),
                 lambda: P.kv_append(w.c, b, k, v, rot=w.rot.cuda().double()),
                 lambda: P.kv_append(w.c, b, k, v, g_k=torch.ones(63, device="cuda")),
                 lambda: P.kv_append(w.c, b, k, v, q_out=q), lambda: P.kv_append(w.c, b, k.cpu(), v),
                 lambda: P.kv_attention(q[..., :32], w.c, b), lambda: P.kv_attention(q, w.c, b, out=q[:2]),
                 lambda: P.kv_attention(q.transpose(0, 1).contiguous().transpose(0, 1), w.c, b),
                 lambda: P.kv_read(w.c, b, dtype=torch.float16),
                 lambda: P.KVBatch(b.ctx_len, b.block_table, b.q_start),
                 lambda: P.KVCache("int8", 128, w.c.k, w.c.v, w.c.k_scale, w.c.v_scale)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: P.kv_attention(w.rows(4, 3), w.c, b), lambda: P.kv_attention(q, w.c, b, window=-1),
                 lambda: P.kv_attention(q, w.c, b, workspace=torch.empty(0, dtype=torch.uint8, device="cuda")),
                 lambda: P.kv_attention(q, w.c, b, out=q), lambda: P.kv_append(w.c, b, k, v, rot=w.rot.cuda()[:63].contiguous())):
        with pytest.raises((P.ProxError, ValueError)):
            call()
    empty = P.KVBatch(b.ctx_len, b.block_table, b.q_start, n_tokens=0)
    assert P.kv_attention(q[:0], w.c, empty).shape == (0, 4, 64)
    assert P.kv_append(w.c, empty, k[:0], v[:0], q=q[:0]).shape == (0, 4, 64)
    assert P.kv_read(w.c, empty)[0].shape == (0, 2, 64)


def test_pages_past_32_bits():
    # 70000 pages of 64 KB: codes past 4 GiB on either side
    import free_ffn_activation_prox_amd as P
    n_pages, KV, hd = 70000, 8, 128
    big = P.KVCache.alloc("int8", n_pages, KV, hd)
    small = World("int8", 16, KV, hd, [150], seed=29, extra=0)
    settle(small, [150])
    where = torch.tensor([n_pages - 1, 66000, 3], dtype=torch.int32)
    b, start = small.batch([150], advance=False)
    far = P.KVBatch(b.ctx_len, where.cuda()[None].contiguous(), b.q_start, n_tokens=150, max_q=150)
    k, v = P.kv_read(small.c, b)
    P.kv_append(big, far, k, v)
    k2, v2 = P.kv_read(big, far, dtype=torch.float32)
    # the values were rounded to bf16 on the way: a step of the new code at most
    assert float((k2 - k.float()).abs().max()) <= 0.51 * float(big.k_scale.max())
    o = small.o
    o2 = KO.Cache("int8", 3, KV, hd)
    sel = where.long().cuda()
    o2.k, o2.v = big.k[sel].cpu().numpy(), big.v[sel].cpu().numpy()
    o2.ks, o2.vs = big.k_scale[sel].cpu().numpy(), big.v_scale[sel].cpu().numpy()
    small.o, small.c, small.table = o2, big, np.array([[0, 1, 2]], np.int32)
    for new in ([1], [150]):
        bb, st = small.batch(new, advance=False)
        bb = P.KVBatch(bb.ctx_len, where.cuda()[None].contiguous(), bb.q_start, n_tokens=bb.n_tokens, max_q=bb.max_q)
        small.attend(bb, st)
    assert not big.k[:3].any() and not big.k[4:66000].any() and not big.v[66001:n_pages - 1].any()


def _step(P, cache, batch, x, rot, H, KV, hd, ws):
    T = x.shape[0]
    q, k, v = x.split([H * hd, KV * hd, KV * hd], 1)
    q = P.kv_append(cache, batch, k.view(T, KV, hd), v.view(T, KV, hd), rot=rot, q=q.view(T, H, hd))
    return P.kv_attention(q, cache, batch, workspace=ws)


def test_steps_together_eager_streams_and_graphs():
    """Append and attention as a decode step runs them: a prompt, then steps;
    eagerly, on a side stream, and as two captured graphs that share one
    workspace, replayed with eager work between.  All agree bit for bit, and
    with the oracle."""
    import free_ffn_activation_prox_amd as P
    H, KV, hd, S = 8, 2, 128, 3
    w = World("int8", H, KV, hd, [400, 300, 200], seed=31)
    rot = w.rot.cuda()
    prompt = [130, 64, 1]
    xs = [bf16(w.rng.standard_normal((n, (H + 2 * KV) * hd))).cuda() for n in (195, 3, 3, 3, 3, 3, 3)]

    def fresh():
        c = P.KVCache("int8", hd, *(torch.from_numpy(a.copy()).cuda() for a in (w.o.k, w.o.v, w.o.ks, w.o.vs)))
        ctx = torch.tensor(prompt, dtype=torch.int32, device="cuda")
        table = torch.from_numpy(w.table).cuda()
        start = torch.tensor([0, 130, 194, 195], dtype=torch.int32, device="cuda")
        return c, ctx, P.KVBatch(ctx, table, start, n_tokens=195, max_q=130), P.KVBatch(ctx, table)

    def run(stream=None):
        c, ctx, first, one = fresh()
        ws = P.alloc_kv_workspace(c, first, H)
        ws1 = P.alloc_kv_workspace(c, one, H)
        outs = [_step(P, c, first, xs[0], rot, H, KV, hd, ws)]
        for x in xs[1:]:
            ctx.add_(1)
            outs.append(_step(P, c, one, x, rot, H, KV, hd, ws1))
        return c, outs

    c0, ref = run()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        c1, got = run()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref, got)) and torch.equal(c0.k, c1.k) and torch.equal(c0.v, c1.v)

    # two graphs of a step on one workspace, replayed in turn
    c2, ctx, first, one = fresh()
    ws1 = P.alloc_kv_workspace(c2, one, H)
    o = _step(P, c2, first, xs[0], rot, H, KV, hd, None)
    assert torch.equal(o, ref[0])
    keep = ctx.clone(), c2.k.clone(), c2.v.clone(), c2.k_scale.clone(), c2.v_scale.clone()
    xin = xs[1].clone()
    warm = torch.cuda.Stream()
    warm.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(warm):
        _step(P, c2, one, xin, rot, H, KV, hd, ws1)
    torch.cuda.current_stream().wait_stream(warm)
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ctx.add_(1)
            y = _step(P, c2, one, xin, rot, H, KV, hd, ws1)
        graphs.append((g, y))
    for t, v in zip((ctx, c2.k, c2.v, c2.k_scale, c2.v_scale), keep):
        t.copy_(v)
    for i, x in enumerate(xs[1:]):
        g, y = graphs[i % 2]
        xin.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, ref[i + 1]), f"replay {i}"
        P.kv_read(c2, one)                    # eager work between the replays
        torch.randn(1000, device="cuda").sum().item()
    assert torch.equal(c2.k, c0.k) and torch.equal(c2.k_scale, c0.k_scale)

    # the oracle over the same steps
    table, ctxs = w.table, np.array(prompt, np.int32)
    rn = w.rot.numpy()
    for i, x in enumerate(xs):
        if i:
            ctxs = ctxs + 1
        start = [0, 130, 194, 195] if i == 0 else None
        mq = 130 if i == 0 else 1
        q, k, v = (f64(t).reshape(x.shape[0], -1, hd) for t in x.split([H * hd, KV * hd, KV * hd], 1))
        KO.append(w.o, table, ctxs, start, mq, k, v, rn)
        qr = np.zeros_like(q)
        for s, row, pos in KO.rows_of(start, ctxs, x.shape[0], mq):
            qr[row] = f64(bf16(KO.turn(q[row], pos, rn, "interleaved", None, 0.0)))
        want, tol = KO.attention(w.o, table, ctxs, start, mq, qr, hd ** -0.5)
        assert np.all(np.abs(f64(ref[i]) - want) <= tol), i


def test_two_streams_at_once_with_their_own_workspaces():
    w = World("fp8", 8, 2, 128, [3000, 2500], seed=37)
    settle(w, [3000, 2500])
    P = w.P
    work = []
    for new in ([1, 1], [300, 200]):
        b, start = w.batch(new, advance=False)
        q = w.rows(b.n_tokens, 8)
        work.append((b, q, w.attend(b, start, q=q)[0], P.alloc_kv_workspace(w.c, b, 8), torch.cuda.Stream()))
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(10):
        for i, (b, q, ref, ws, s) in enumerate(work):
            outs[i].append(P.kv_attention(q, w.c, b, workspace=ws, stream=s, out=torch.empty_like(q)))
    torch.cuda.synchronize()
    for i, (b, q, ref, ws, s) in enumerate(work):
        assert all(torch.equal(o, ref) for o in outs[i])


def test_given_stream_owns_what_the_call_allocates():
    # calls on a side stream, their workspace and outputs allocated by the calls,
    # while the current stream allocates and writes memory of the same sizes
    w = World("int8", 8, 2, 128, [4000, 900], seed=47)
    settle(w, [4000, 900])
    P = w.P
    b, start = w.batch([1, 1], advance=False)
    q = w.rows(2, 8)
    ref, _ = w.attend(b, start, q=q)
    kr, vr = P.kv_read(w.c, b)
    n = P.kv_workspace_bytes(w.c, b, 8)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    outs = []
    for i in range(30):
        outs.append((P.kv_attention(q, w.c, b, stream=side), *P.kv_read(w.c, b, stream=side)))
        junk = [torch.full((n + 256,), 0xff, dtype=torch.uint8, device="cuda") for _ in range(2)]
        del junk
    torch.cuda.synchronize()
    assert all(torch.equal(o, ref) and torch.equal(k, kr) and torch.equal(v, vr) for o, k, v in outs)


def test_many_sequences():
    # more tiles of rows than a wave sees at once; lengths from 0 on, the same pages read by two sequences
    rng = np.random.default_rng(43)
    lens = [int(n) for n in rng.integers(0, 150, 150)]
    w = World("int8", 4, 2, 64, [max(n, 1) for n in lens], seed=43)
    settle(w, lens)
    w.table[7] = w.table[3]
    w.ctx[7] = w.ctx[3]
    b, start = w.batch([1] * 150, advance=False)
    w.attend(b, start)
    new = [int(min(n, k)) for n, k in zip(lens, rng.integers(0, 40, 150))]
    new[7] = min(new[7], int(w.ctx[7]))
    b, start = w.batch(new, advance=False)
    w.attend(b, start)
    w.attend(b, start, window=20)


@pytest.mark.parametrize("kind,H,KV,hd", [("int8", 8, 2, 64), ("fp8", 9, 3, 128)])
def test_long_chunks_among_many_short_sequences(kind, H, KV, hd):
    # sequences of few tokens and longer ones get launches of their own here: 0 and 1 tokens, the last
    # number that counts as few and the first that does not, long contexts on both sides
    rng = np.random.default_rng(H)
    few = 16 // (H // KV)
    lens = [int(n) for n in rng.integers(1, 130, 140)]
    lens[5], lens[77], lens[139] = 5000, 1500, 200
    w = World(kind, H, KV, hd, lens, seed=H)
    settle(w, lens)
    new = [int(min(n, k)) for n, k in zip(lens, rng.choice([0, 1, 1, 1, 2, few, few + 1, 20], 140))]
    new[5], new[77], new[139] = 1, 700, 130
    b, start = w.batch(new, advance=False, pad=3)
    w.attend(b, start)
    w.attend(b, start, window=100)
    # a captured call follows the lengths: only short ones, only long ones, both again
    q = w.rows(b.n_tokens, H, 1.5)
    out = torch.zeros_like(q)
    ws = w.P.alloc_kv_workspace(w.c, b, H)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        w.P.kv_attention(q, w.c, b, out=out, workspace=ws)
    for keep in (lambda n: n <= few, lambda n: n > few, lambda n: True):
        now = [n if keep(n) else 0 for n in new]
        begin = np.concatenate([[0], np.cumsum(now)]).astype(np.int32)
        b.q_start.copy_(torch.from_numpy(begin))
        out.fill_(7.0)
        g.replay()
        torch.cuda.synchronize()
        want, tol = KO.attention(w.o, w.table, w.ctx, begin, b.max_q, f64(q), hd ** -0.5, 0)
        got, idle = f64(out), np.isnan(want).all((1, 2))
        assert np.array_equal(got[idle], np.full_like(got[idle], 7.0))
        assert (np.abs(got[~idle] - want[~idle]) <= tol[~idle]).all()


@pytest.mark.parametrize("kind,hd", [("int8", 64), ("fp8", 128)])
def test_append_and_read_of_a_long_chunk_among_many_short_sequences(kind, hd):
    # more than 64 sequences, of which one has many pages: blocks find their pages in the lengths
    lens = [1 + (7 * s) % 130 for s in range(140)]
    w = World(kind, 4, 2, hd, [n + 40 for n in lens[:99]] + [1200] + [n + 40 for n in lens[100:]], seed=hd)
    settle(w, lens)
    w.append([s % 3 for s in range(99)] + [1000] + [1] * 40, norm=True, pad=2)
    w.table[3, 0] = -1
    w.ctx[100] = 0                                     # its row has no position
    new = [s % 4 for s in range(99)] + [900] + [1] * 40
    b, start = w.batch([min(n, 1000) for n in new], advance=False, pad=3)
    ko, vo = (torch.full((b.n_tokens, 2, hd), 7.0, dtype=torch.float32, device="cuda") for _ in range(2))
    w.P.kv_read(w.c, b, dtype=torch.float32, k_out=ko, v_out=vo)
    kw, vw = (np.full((b.n_tokens, 2, hd), 7.0) for _ in range(2))
    for s, row, pos in KO.rows_of(start, w.ctx, b.n_tokens, b.max_q):
        kw[row] = vw[row] = 0
        if pos >= 0:
            k, v, there = KO.gather(w.o, w.table, s, pos, pos + 1)
            if there[0]:
                kw[row], vw[row] = k[0].astype(np.float32), v[0].astype(np.float32)
    assert np.array_equal(f64(ko), kw) and np.array_equal(f64(vo), vw)
