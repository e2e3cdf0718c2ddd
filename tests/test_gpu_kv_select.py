"""Bounds of keys and selection of pages against the oracle: whole numbers, so
every bound and every listed page is equal."""

import numpy as np
import pytest
import torch

from oracle import kv_ops_oracle as OO
from test_gpu_kv import World, bf16, f64, settle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def bounds_of(w, new=None, max_q=None, out=None):
    """Bounds over the last new[s] tokens (default all) on the GPU, checked against the oracle's."""
    new = list(w.ctx) if new is None else new
    b, start = w.batch(new, advance=False, max_q=max_q)
    if out is None:
        out = w.P.alloc_kv_bounds(w.c)
    exp = out.cpu().numpy()
    got = w.P.kv_page_bounds(w.c, b, out)
    torch.cuda.synchronize()
    assert got is out
    OO.bounds(w.o, w.table, w.ctx, start, b.n_tokens, b.max_q, exp)
    assert np.array_equal(out.cpu().numpy(), exp)
    return out


def chosen(w, bnd, new, keep, first=1, last=1, q=None, pad=0, max_q=None, packed=False):
    b, start = w.batch(new, advance=False, pad=pad, max_q=max_q)
    T = b.n_tokens
    if q is None:
        q = bf16(w.rng.standard_normal((T, w.H, w.hd)) * np.exp(0.7 * w.rng.standard_normal((1, w.H, 1)))).cuda()
    if packed:
        big = torch.zeros(T, (w.H + 1) * w.hd, dtype=torch.bfloat16, device="cuda")
        big[:, :w.H * w.hd] = q.view(T, -1)
        q = big[:, :w.H * w.hd].view(T, w.H, w.hd)
    pages = torch.full((T, w.KV, keep), -7, dtype=torch.int32, device="cuda")
    got = w.P.kv_select(q, w.c, b, bnd, keep, first=first, last=last, pages=pages)
    torch.cuda.synchronize()
    assert got is pages
    exp = np.full((T, w.KV, keep), -7, np.int32)
    OO.select(w.o, w.table, w.ctx, start, b.max_q, f64(q), bnd.cpu().numpy(), keep, first, last, exp)
    got = got.cpu().numpy()
    bad = np.argwhere((got != exp).any(-1))
    assert bad.size == 0, f"row, head {bad[:3].tolist()}: {got[tuple(bad[0])][:20]} for {exp[tuple(bad[0])][:20]}"
    return exp


CASES = [("int8", 4, 2, 64), ("fp8", 6, 6, 128), ("int8", 7, 1, 80), ("fp8", 2, 2, 96), ("int8", 3, 3, 8),
         ("fp8", 5, 1, 16), ("int8", 2, 1, 256), ("fp8", 20, 1, 192), ("int8", 34, 2, 64)]


@pytest.mark.parametrize("kind,H,KV,hd", CASES)
def test_bounds_over_several_calls(kind, H, KV, hd):
    w = World(kind, H, KV, hd, [300, 64, 1, 130], seed=hd)
    out = None
    for new in ([1, 0, 0, 60], [130, 64, 1, 4], [1, 0, 0, 1]):
        w.append(new, rotate=False)
        out = bounds_of(w, new, out=out)
    bounds_of(w)


def test_bounds_of_any_bytes():
    # codes that no append writes: -128, and e4m3 NaN
    for kind in ("int8", "fp8"):
        w = World(kind, 2, 2, 64, [256, 70], seed=3)
        w.ctx[:] = [256, 70]
        bounds_of(w)
        bounds_of(w, [3, 1], max_q=2)                   # a row beyond max_q is no token of the call


def test_bounds_of_pages_and_positions_that_do_not_exist():
    w = World("int8", 2, 1, 64, [192, 192, 192], seed=5)
    w.table[1, 1] = w.o.n_pages
    w.table[2, 0] = -5
    w.ctx[:] = [220, 150, 100]
    bounds_of(w)
    w.ctx[:] = [-40, 5, 0]
    bounds_of(w, [30, 20, 3])


@pytest.mark.parametrize("kind,H,KV,hd", CASES)
def test_selected_pages(kind, H, KV, hd):
    w = World(kind, H, KV, hd, [1500, 64, 3, 700], seed=hd + 1)
    settle(w, [1500, 64, 3, 700])
    bnd = bounds_of(w)
    chosen(w, bnd, [1, 1, 1, 1], 5)
    chosen(w, bnd, [1, 0, 2, 70], 4, first=0, last=2, pad=3, packed=True)
    chosen(w, bnd, [300, 64, 3, 5], 7, first=2, last=3)
    chosen(w, bnd, [1, 1, 1, 1], 1, first=0, last=1)
    chosen(w, bnd, [1, 1, 1, 1], 40)                    # more than there are
    chosen(w, bnd, [20, 7, 0, 0], 3, max_q=9)


def test_without_q_start():
    w = World("int8", 8, 2, 128, [900, 100, 500], seed=8)
    settle(w, [900, 100, 500])
    bnd = bounds_of(w)
    P = w.P
    b = P.KVBatch(torch.from_numpy(w.ctx.copy()).cuda(), torch.from_numpy(w.table).cuda())
    q = w.rows(3, 8, 2.0)
    got = P.kv_select(q, w.c, b, bnd, 6)
    exp = np.zeros((3, 2, 6), np.int32)
    OO.select(w.o, w.table, w.ctx, None, 1, f64(q), bnd.cpu().numpy(), 6, 1, 1, exp)
    assert np.array_equal(got.cpu().numpy(), exp)


def test_many_pages_and_ties():
    # 300 and more pages of few different bounds: whole runs of equal keys
    for kind in ("int8", "fp8"):
        w = World(kind, 4, 1, 64, [64 * 333 - 9], seed=11)
        w.ctx[:] = [64 * 333 - 9]
        bnd = torch.from_numpy(w.rng.integers(-2, 3, (w.o.n_pages, 1, 2, 64)).astype(np.int8)).cuda()
        bnd[:, :, :, 4:] = 0
        w.o.ks[:] = 0.5
        w.c.k_scale.fill_(0.5)
        q = bf16(np.sign(w.rng.standard_normal((5, 4, 64)))).cuda()
        for keep in (1, 2, 64, 65, 200, 332, 333, 334):
            chosen(w, bnd, [5], keep, first=min(1, keep - 1), q=q)


def test_long_context():
    # more pages than threads, several rows of one block
    w = World("int8", 8, 1, 64, [64 * 2500], seed=12, extra=0)
    w.ctx[:] = [64 * 2500 - 70]
    bnd = torch.from_numpy(w.rng.integers(-127, 128, (w.o.n_pages, 1, 2, 64)).astype(np.int8)).cuda()
    chosen(w, bnd, [1], 64)
    chosen(w, bnd, [3], 1200, first=3, last=7)


@pytest.mark.parametrize("pages,H,kinds", [(400, 3, 200), (700, 8, 3), (1500, 20, 200), (2048, 1, 1), (2049, 2, 4)])
def test_tables_of_any_width(pages, H, kinds):
    """Rows selected by a wave (of 8 or 32 keys a lane) and by a block, from few and many different keys."""
    w = World("int8", H, 1, 64, [64 * pages, 64 * 70], seed=pages, extra=0)
    w.ctx[:] = [64 * pages - 5, 64 * 70 - 1]
    bnd = torch.from_numpy(w.rng.integers(0, kinds, (w.o.n_pages, 1, 2, 64)).astype(np.int64) - kinds // 2).to(torch.int8).cuda()
    w.o.ks[:] = w.rng.choice(np.float32([0.5, 1.0]), w.o.ks.shape)
    w.c.k_scale.copy_(torch.from_numpy(w.o.ks))
    chosen(w, bnd, [1, 1], 33)
    chosen(w, bnd, [5, 70], 100, first=2, last=3)
    chosen(w, bnd, [9, 0], 3 * pages // 4)
    chosen(w, bnd, [2, 3], 2)


def test_workspace_of_any_content_twice():
    w = World("int8", 8, 2, 64, [64 * 900], seed=19, extra=0)
    w.ctx[:] = [64 * 900 - 5]
    bnd = torch.from_numpy(w.rng.integers(-127, 128, (w.o.n_pages, 2, 2, 64)).astype(np.int8)).cuda()
    P = w.P
    b, _ = w.batch([2], advance=False)
    q = w.rows(2, 8)
    ws = P.alloc_kv_select_workspace(w.c, b, 8)
    assert ws.numel() > 256                                # several blocks a row
    got = []
    for fill in (0, 0xff, 0x5a):
        ws.fill_(fill)
        got += [P.kv_select(q, w.c, b, bnd, 40, workspace=ws) for _ in range(3)]
    assert all(torch.equal(g, got[0]) for g in got)


def test_infinities_nan_zeros_and_tiny_values():
    w = World("int8", 4, 2, 64, [900], seed=13)
    settle(w, [900])
    bnd = bounds_of(w)
    q = bf16(w.rng.standard_normal((8, 4, 64)))
    q[0] = 0
    q[1, 0, 3], q[1, 1, 4] = float("inf"), float("-inf")
    q[2, 2, 5] = float("nan")
    q[3] = float("nan")
    q[4] = float("inf")
    q[5] *= 2.0 ** -126
    q[6] *= 2.0 ** 120
    q[7, :, 0] = 1e38
    chosen(w, bnd, [8], 4, q=q.cuda())
    # page scales that no append writes
    w.o.ks[w.table[0, 3]] = np.inf
    w.o.ks[w.table[0, 4]] = np.nan
    w.o.ks[w.table[0, 5]] = 0
    w.o.ks[w.table[0, 6]] = 1e-40
    w.c.k_scale.copy_(torch.from_numpy(w.o.ks))
    chosen(w, bnd, [8], 6, first=0, q=q.cuda())


def test_pages_and_positions_that_do_not_exist():
    w = World("fp8", 4, 2, 64, [900, 300, 300], seed=14)
    settle(w, [900, 300, 300])
    bnd = bounds_of(w)
    w.table[0, [0, 5, 14]] = [-1, w.o.n_pages, -9]      # among them the first and a row's own
    w.table[1] = -1
    w.ctx[:] = [64 * w.table.shape[1] + 3, 300, 2]      # rows behind the table, and before position 0
    chosen(w, bnd, [80, 2, 5], 6)
    chosen(w, bnd, [80, 2, 5], 20)


def test_captured_and_replayed_with_moving_lengths():
    w = World("int8", 8, 2, 128, [2000, 700], seed=15)
    settle(w, [1900, 600])
    P = w.P
    ctx = torch.from_numpy(w.ctx.copy()).cuda()
    table = torch.from_numpy(w.table).cuda()
    b = P.KVBatch(ctx, table)
    bnd = bounds_of(w)
    q, k, v = w.rows(2, 8), w.rows(2, 2), w.rows(2, 2)
    pages = torch.zeros(2, 2, 5, dtype=torch.int32, device="cuda")

    def step():
        ctx.add_(1)
        P.kv_append(w.c, b, k, v)
        P.kv_page_bounds(w.c, b, bnd)
        P.kv_select(q, w.c, b, bnd, 5, pages=pages)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        step()
    for i in range(70):
        q.copy_(w.rows(2, 8))
        k.copy_(w.rows(2, 2))
        g.replay()
        if i % 9 == 0:
            torch.cuda.synchronize()
            bh, ph = bnd.clone(), pages.clone()
            w.ctx = ctx.cpu().numpy().copy()
            P.kv_page_bounds(w.c, P.KVBatch(ctx, table, torch.tensor([0, w.ctx[0], w.ctx.sum()], dtype=torch.int32, device="cuda"),
                                            n_tokens=int(w.ctx.sum()), max_q=int(w.ctx.max())), bnd)
            assert torch.equal(bh, bnd), i               # the touched pages' bounds were up to date
            w.o.ks = w.c.k_scale.cpu().numpy()
            exp = np.zeros((2, 2, 5), np.int32)
            OO.select(w.o, w.table, w.ctx, None, 1, f64(q), bnd.cpu().numpy(), 5, 1, 1, exp)
            assert np.array_equal(ph.cpu().numpy(), exp), i


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_bounds_of_a_page_that_one_of_its_sequences_is_cut_back_into(kind):
    """The calls that the header allows keep the bounds of all that a holder of the page has in it: the rows of
    kv_pages name no token of the sequence that was cut back, until it holds the page alone."""
    w = World(kind, 2, 1, 64, [200, 200], seed=21, extra=4)
    P = w.P
    pool = P.KVPool.alloc(w.o.n_pages, 2, w.table.shape[1])
    bnd = P.alloc_kv_bounds(w.c)
    dev = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731

    def call(*want, parent=None, shared=None, refused=0):
        start, _, status = P.kv_pages(pool, dev(*want), 400, parent=parent, shared=shared)
        assert status.tolist()[0] == refused
        b = P.KVBatch(pool.ctx_len, pool.block_table, start, n_tokens=400, max_q=400)
        k = w.rows(400, 1)
        P.kv_append(w.c, b, k, w.rows(400, 1))
        P.kv_page_bounds(w.c, b, bnd)
        torch.cuda.synchronize()

    def holds(seq, tokens):
        """Bounds of the sequence's pages are the oracle's over its tokens."""
        w.o.k, w.o.ks = w.c.k.cpu().numpy().reshape(w.o.k.shape), w.c.k_scale.cpu().numpy()
        table, got = pool.block_table.cpu().numpy()[seq:seq + 1], bnd.cpu().numpy()
        exp = got.copy()
        OO.bounds(w.o, table, np.array([tokens]), np.array([0, tokens]), tokens, tokens, exp)
        for page in table[0, :-(-tokens // 64)]:
            assert np.array_equal(got[page], exp[page])

    call(128, 0)
    call(130, 128, parent=dev(-1, 0), shared=dev(0, 2))
    holds(0, 130)
    call(131, 100)                                                 # cut back into a page that sequence 0 has in full
    call(132, 101, refused=1)
    assert pool.ctx_len.tolist() == [132, 100]
    holds(0, 132)
    call(0, 100)                                                   # sequence 1 has the page alone: it goes on there
    call(0, 103)
    holds(1, 103)
