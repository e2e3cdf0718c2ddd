"""Attention over selected pages against the oracle: the bound that
``kv_oracle.attention`` derives, for every row over the pages that it lists."""

import numpy as np
import pytest
import torch

from oracle import kv_ops_oracle as OO
from test_gpu_kv import World, f64, settle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def lists(w, start, T, keep, full=False):
    """Random ascending pages of what each row sees, the row's own often among them."""
    out = np.full((T, w.KV, keep), -1, np.int32)
    for s in range(len(w.ctx)):
        for row in range(start[s], start[s + 1]):
            n = max(0, (int(w.ctx[s]) - int(start[s + 1]) + row) // 64 + 1)
            for h in range(w.KV):
                k = min(keep, n) if full else int(w.rng.integers(0, min(keep, n) + 1))
                out[row, h, :k] = np.sort(w.rng.permutation(n)[:k])
    return out


def attend(w, new, pages=None, keep=4, q=None, scale=None, pad=0, max_q=None, packed=False, **kw):
    b, start = w.batch(new, advance=False, pad=pad, max_q=max_q)
    T = b.n_tokens
    q = w.rows(T, w.H, 1.5) if q is None else q
    if packed:
        big = torch.zeros(T, w.H * w.hd + 16, dtype=torch.bfloat16, device="cuda")
        big[:, :w.H * w.hd] = q.view(T, -1)
        q = big[:, :w.H * w.hd].view(T, w.H, w.hd)
    if pages is None:
        pages = lists(w, start, T, keep)
    out = torch.full((T, w.H, w.hd), 7.0, dtype=torch.bfloat16, device="cuda")
    w.P.kv_attention_selected(q, w.c, b, torch.from_numpy(pages).cuda(), out=out, scale=scale, **kw)
    torch.cuda.synchronize()
    want, tol = OO.attention_selected(w.o, w.table, w.ctx, start, b.max_q, f64(q), pages, w.hd ** -0.5 if scale is None else scale)
    got = f64(out)
    idle = np.isnan(want).all((1, 2))
    assert np.array_equal(got[idle], np.full_like(got[idle], 7.0)), "rows outside the sequences were written"
    err = np.abs(got[~idle] - want[~idle])
    worst = float(np.max(err / tol[~idle].clip(1e-37))) if err.size else 0.0
    assert np.isfinite(got[~idle]).all() and worst <= 1.0, f"error {worst:.3f} of the bound"
    return out


CASES = [("int8", 4, 2, 64), ("fp8", 6, 6, 128), ("int8", 7, 1, 80), ("fp8", 2, 2, 96), ("int8", 3, 3, 8),
         ("fp8", 5, 1, 16), ("int8", 2, 1, 256), ("fp8", 20, 1, 192), ("int8", 34, 2, 64), ("int8", 16, 1, 256)]


@pytest.mark.parametrize("kind,H,KV,hd", CASES)
def test_against_oracle(kind, H, KV, hd):
    w = World(kind, H, KV, hd, [1500, 64, 3, 700], seed=hd + 2)
    settle(w, [1500, 64, 3, 700])
    attend(w, [1, 1, 1, 1], keep=6)
    attend(w, [1, 0, 2, 9], keep=1, pad=3, packed=True)
    attend(w, [5, 64, 3, 5], keep=24)
    attend(w, [20, 7, 0, 0], keep=30, max_q=9)
    attend(w, [0, 1, 0, 0], keep=3, scale=-0.2)
    attend(w, [1, 1, 0, 0], keep=3, scale=0.0)


def test_many_sequences_with_empty_ones_between():
    """Selection and attention where a row's sequence is one of hundreds, of which many have no rows."""
    n = 333
    w = World("int8", 4, 2, 64, [200] * n, seed=27)
    settle(w, [int(x) for x in w.rng.integers(1, 200, n)])
    full, _ = w.batch([int(c) for c in w.ctx], advance=False)
    bnd = w.P.kv_page_bounds(w.c, full, w.P.alloc_kv_bounds(w.c))
    for most in (1, 3):
        new = [int(min(c, x)) for c, x in zip(w.ctx, w.rng.integers(-1, most + 1, n).clip(0))]
        b, start = w.batch(new, advance=False, pad=5)
        q = w.rows(b.n_tokens, 4, 1.5)
        pages = torch.full((b.n_tokens, 2, 2), -7, dtype=torch.int32, device="cuda")
        w.P.kv_select(q, w.c, b, bnd, 2, first=0, pages=pages)
        exp = np.full((b.n_tokens, 2, 2), -7, np.int32)
        OO.select(w.o, w.table, w.ctx, start, b.max_q, f64(q), bnd.cpu().numpy(), 2, 0, 1, exp)
        assert np.array_equal(pages.cpu().numpy(), exp)
        attend(w, new, pages=exp, q=q, pad=5)


def test_without_q_start_and_more_entries_than_pages():
    w = World("int8", 8, 2, 128, [900, 100, 500], seed=8)
    settle(w, [900, 100, 500])
    P = w.P
    b = P.KVBatch(torch.from_numpy(w.ctx.copy()).cuda(), torch.from_numpy(w.table).cuda())
    q = w.rows(3, 8, 1.5)
    pages = lists(w, [0, 1, 2, 3], 3, 200, full=True)
    out = f64(P.kv_attention_selected(q, w.c, b, torch.from_numpy(pages).cuda()))
    want, tol = OO.attention_selected(w.o, w.table, w.ctx, None, 1, f64(q), pages, 128 ** -0.5)
    assert (np.abs(out - want) <= tol).all()


def test_every_page_listed_is_the_attention_over_all():
    for kind in ("int8", "fp8"):
        w = World(kind, 8, 2, 64, [1000, 130], seed=21)
        settle(w, [1000, 130])
        b, start = w.batch([3, 70], advance=False)
        q = w.rows(73, 8, 1.5)
        pages = lists(w, start, 73, 16, full=True)
        attend(w, [3, 70], pages=pages, q=q)
        w.attend(b, start, q=q)


def test_lists_of_any_content():
    w = World("fp8", 4, 2, 64, [900, 300], seed=22)
    settle(w, [900, 300])
    odd = np.array([[3, 3, 5, 4, 6, 2 ** 31 - 1, -2 ** 31, 7], [-1, -1, 2, -1, 3, 3, 1, 2], [14, 13, 12, 11, 10, 9, 8, 7],
                    [15, 14, 0, 1, 100, 14, 13, -1]], np.int32)
    pages = np.stack([odd[[i % 4, (i + 1) % 4]] for i in range(10)])
    attend(w, [6, 4], pages=pages)
    attend(w, [10, 0], pages=w.rng.integers(-3, 20, (10, 2, 100)).astype(np.int32))


def test_pages_and_positions_that_do_not_exist():
    for kind in ("int8", "fp8"):
        w = World(kind, 4, 2, 64, [900, 300, 300], seed=14)
        settle(w, [900, 300, 300])
        w.table[0, [0, 5, 14]] = [-1, w.o.n_pages, -9]
        w.table[1] = -1
        w.ctx[:] = [64 * w.table.shape[1] + 3, 300, 2]
        attend(w, [80, 2, 5], keep=6)
        attend(w, [80, 2, 5], pages=np.tile(np.arange(20, dtype=np.int32), (87, 2, 1)))


def test_unlike_value_scales_and_large_scores():
    w = World("int8", 8, 1, 128, [2000], seed=23)
    settle(w, [2000])
    w.o.vs *= np.exp2(w.rng.integers(-90, 90, w.o.vs.shape)).astype(np.float32)
    w.c.v_scale.copy_(torch.from_numpy(w.o.vs))
    attend(w, [4], keep=32)
    w.o.ks *= np.float32(64.0)
    w.c.k_scale.copy_(torch.from_numpy(w.o.ks))
    attend(w, [4], keep=32)


@pytest.mark.parametrize("T,keep", [(1, 64), (1, 300), (3, 129), (40, 17), (300, 8)])
def test_splits(T, keep):
    """Blocks a row from many to one; longer lists than a wave looks at once."""
    w = World("int8", 8, 2, 64, [64 * 400], seed=T, extra=0)
    w.ctx[:] = [64 * 400 - 20]
    w.o.ks[:], w.o.vs[:] = 0.01, 0.01
    w.c.k_scale.fill_(0.01), w.c.v_scale.fill_(0.01)
    _, start = w.batch([T], advance=False)
    pages = lists(w, start, T, keep, full=True)
    attend(w, [T], pages=pages)


def test_same_result_twice_and_workspace_of_any_content():
    w = World("int8", 8, 2, 128, [3000], seed=24)
    settle(w, [3000])
    b, start = w.batch([1], advance=False)
    q, pages = w.rows(1, 8, 1.5), torch.from_numpy(lists(w, start, 1, 40, full=True)).cuda()
    ws = w.P.alloc_kv_selected_workspace(w.c, b, 8, 40)
    got = []
    for fill in (0, 0xff, 0x5a):
        ws.fill_(fill)
        got += [w.P.kv_attention_selected(q, w.c, b, pages, workspace=ws) for _ in range(3)]
    assert all(torch.equal(g, got[0]) for g in got)


def test_two_captured_graphs_share_a_workspace():
    w = World("fp8", 8, 2, 64, [2000, 2000], seed=25)
    settle(w, [2000, 1500])
    P = w.P
    ctx, table = torch.from_numpy(w.ctx.copy()).cuda(), torch.from_numpy(w.table).cuda()
    b = P.KVBatch(ctx, table)
    bnd = P.alloc_kv_bounds(w.c)
    P.kv_page_bounds(w.c, P.KVBatch(ctx, table, torch.tensor([0, 2000, 3500], dtype=torch.int32, device="cuda"),
                                    n_tokens=3500, max_q=2000), bnd)
    q = w.rows(2, 8, 1.5)
    ws = P.alloc_kv_selected_workspace(w.c, b, 8, 20)
    graphs, outs = [], []
    for keep in (20, 9):
        pages = torch.empty(2, 2, keep, dtype=torch.int32, device="cuda")
        out = torch.empty_like(q)

        def step():
            P.kv_select(q, w.c, b, bnd, keep, pages=pages)
            P.kv_attention_selected(q, w.c, b, pages, out=out, workspace=ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
        outs.append((keep, out))
    for i in range(8):
        q.copy_(w.rows(2, 8, 1.5))
        for g in graphs if i % 2 else graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for keep, out in outs:
            assert torch.equal(out, P.kv_attention_selected(q, w.c, b, P.kv_select(q, w.c, b, bnd, keep))), (i, keep)


def test_memory_let_go_before_the_stream_runs():
    w = World("int8", 8, 2, 128, [900, 700], seed=26)
    settle(w, [900, 700])
    P = w.P
    b, start = w.batch([2, 1], advance=False)
    bnd = P.alloc_kv_bounds(w.c)
    full, _ = w.batch([900, 700], advance=False)
    P.kv_page_bounds(w.c, full, bnd)
    q = w.rows(3, 8, 1.5)
    want = P.kv_attention_selected(q, w.c, b, P.kv_select(q, w.c, b, bnd, 5))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)      # the calls below wait behind this

    def calls():
        batch = P.KVBatch(b.ctx_len.clone(), b.block_table.clone(), b.q_start.clone(), n_tokens=3, max_q=2)
        qq, bb = q.clone(), torch.zeros_like(bnd)
        fb = P.KVBatch(full.ctx_len.clone(), full.block_table.clone(), full.q_start.clone(), n_tokens=1600, max_q=900)
        side.wait_stream(torch.cuda.current_stream())
        P.kv_page_bounds(w.c, fb, bb, stream=side)
        pages = P.kv_select(qq, w.c, batch, bb, 5, stream=side)
        out = P.kv_attention_selected(qq, w.c, batch, pages, stream=side)
        return out, {t.data_ptr() for t in (qq, bb, pages, batch.ctx_len, batch.block_table, batch.q_start)}, \
            [t.nbytes for t in (qq, bb, batch.block_table, fb.q_start)]
    out, kept, sizes = calls()
    assert not side.query()
    junk = [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for n in sizes + [8, 12] for _ in range(2)]
    again = {t.data_ptr() for t in junk}
    assert not side.query() and not kept & again
    torch.cuda.synchronize()
    assert torch.equal(out, want)
