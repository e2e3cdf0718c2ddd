"""Attention with a shared prefix against the oracle: the bound that
``kv_oracle.attention`` derives, over the pages that each sequence sees.

The bound holds as it is: a row's sums are those over its pages, and that they are
put together from two launches is one join of parts more, among the 20 roundings
that it counts for all that happens once."""

import numpy as np
import pytest
import torch

from oracle import kv_oracle as KO
from oracle import kv_ops_oracle as OO
from test_gpu_kv import World, f64, settle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def attend(w, new, shared, groups=None, q=None, scale=None, pad=0, max_q=None, packed=False, **kw):
    b, start = w.batch(new, advance=False, pad=pad, max_q=max_q)
    T = b.n_tokens
    q = w.rows(T, w.H, 1.5) if q is None else q
    if packed:
        big = torch.zeros(T, w.H * w.hd + 16, dtype=torch.bfloat16, device="cuda")
        big[:, :w.H * w.hd] = q.view(T, -1)
        q = big[:, :w.H * w.hd].view(T, w.H, w.hd)
    out = torch.full((T, w.H, w.hd), 7.0, dtype=torch.bfloat16, device="cuda")
    w.P.kv_attention_shared(q, w.c, b, dev(shared), group_start=dev(groups), out=out, scale=scale, **kw)
    torch.cuda.synchronize()
    want, tol = OO.attention_shared(w.o, w.table, w.ctx, start, b.max_q, f64(q), shared, groups,
                                    w.hd ** -0.5 if scale is None else scale)
    got = f64(out)
    idle = np.ones(T, bool)
    idle[[row for _, row, _ in KO.rows_of(start, w.ctx, T, b.max_q)]] = False
    assert np.array_equal(got[idle], np.full_like(got[idle], 7.0)), "rows outside the sequences were written"
    got, want, tol = got[~idle], want[~idle], tol[~idle]
    assert np.array_equal(np.isnan(got), np.isnan(want))             # e4m3 NaN codes among random bytes
    err = np.abs(got - want)[~np.isnan(want)]
    worst = float(np.max(err / tol[~np.isnan(want)].clip(1e-37))) if err.size else 0.0
    assert np.isfinite(err).all() and worst <= 1.0, f"error {worst:.3f} of the bound"
    return out


def share(w, groups, shared):
    """Entries of the shared pages of all but each group's first sequence name no page: nothing reads them."""
    for (a, b), p in zip(zip(groups, groups[1:]), shared):
        w.table[a + 1:b, :p] = -1


CASES = [("int8", 4, 2, 64), ("fp8", 6, 6, 128), ("int8", 7, 1, 80), ("fp8", 2, 2, 96), ("int8", 3, 3, 8),
         ("fp8", 5, 1, 16), ("int8", 2, 1, 256), ("fp8", 20, 1, 192), ("int8", 34, 2, 64)]


@pytest.mark.parametrize("kind,H,KV,hd", CASES)
def test_against_oracle(kind, H, KV, hd):
    w = World(kind, H, KV, hd, [700, 500, 449, 900, 300], seed=hd + 3)
    settle(w, [700, 500, 449, 900, 300])
    share(w, [0, 3, 5], [7, 3])
    attend(w, [1, 1, 1, 1, 1], [7, 3], [0, 3, 5])
    attend(w, [3, 0, 1, 70, 40], [7, 3], [0, 3, 5], pad=4, packed=True)
    attend(w, [3, 5, 1, 70, 90], [6, 3], [0, 3, 5], max_q=20)
    attend(w, [0, 1, 1, 2, 0], [7, 3], [0, 3, 5], scale=-0.2)


def test_one_group_without_q_start():
    for kind in ("int8", "fp8"):
        w = World(kind, 8, 2, 128, [900] * 5, seed=31)
        settle(w, [900, 513, 600, 700, 577])
        share(w, [0, 5], [8])
        P = w.P
        b = P.KVBatch(torch.from_numpy(w.ctx.copy()).cuda(), torch.from_numpy(w.table).cuda())
        q = w.rows(5, 8, 1.5)
        out = f64(P.kv_attention_shared(q, w.c, b, dev([8])))
        want, tol = OO.attention_shared(w.o, w.table, w.ctx, None, 1, f64(q), [8], None, 128 ** -0.5)
        assert (np.abs(out - want) <= tol).all()


def test_many_sequences_and_tiles():
    # more rows than a tile of 256; more sequences than a wave looks at once
    w = World("int8", 8, 2, 64, [64 * 6] + [64 * 6] * 79, seed=32)
    settle(w, [64 * 6] + [int(x) for x in w.rng.integers(64 * 4 + 1, 64 * 6, 79)])
    share(w, [0, 80], [4])
    attend(w, [1] * 80, [4])
    new = [int(min(c - 256, n)) for c, n in zip(w.ctx, w.rng.integers(0, 9, 80))]
    attend(w, new, [4])


def test_sequences_that_share_nothing():
    w = World("int8", 4, 2, 64, [500, 100, 300, 500, 200, 128], seed=33)
    settle(w, [500, 100, 300, 500, 200, 128])
    # inside the prefix (1), at its end (5: its first row is at 127 < 128), outside every group (0, 4), shared 0 (3)
    for groups, shared in (([1, 3, 4], [4, 0]), ([2, 6], [2]), ([0, 6], [0]), ([0, 1, 1, 6], [3, 5, 0])):
        attend(w, [1, 1, 1, 1, 1, 1], shared, groups)
        attend(w, [20, 50, 3, 300, 0, 1], shared, groups)


def test_a_group_of_one_is_the_attention_over_all():
    w = World("fp8", 8, 2, 64, [2000], seed=34)
    settle(w, [2000])
    b, start = w.batch([37], advance=False)
    q = w.rows(37, 8, 1.5)
    attend(w, [37], [30], q=q)
    attend(w, [37], [1], q=q)
    attend(w, [37], [10 ** 6], q=q)        # more than there are pages: inside the prefix
    w.attend(b, start, q=q)


def test_pages_and_positions_that_do_not_exist():
    for kind in ("int8", "fp8"):
        w = World(kind, 4, 2, 64, [900, 300, 300], seed=35)
        settle(w, [900, 300, 300])
        w.table[0, [0, 2, 14]] = [-1, w.o.n_pages, -9]
        w.ctx[:] = [64 * w.table.shape[1] + 3, 300, 64 * w.table.shape[1] + 1]
        for sh in (1, 3, 4):
            attend(w, [8, 2, 5], [sh])
        w.ctx[:] = [-40, 5, 0]
        attend(w, [30, 20, 3], [2])
        w.table[:] = -1
        w.ctx[:] = [900, 300, 290]
        attend(w, [3, 3, 1], [4])


def test_groups_of_any_content_stay_in_bounds():
    """Groups that do not rise, overlap or leave the batch name rows and pages of the batch
    all the same; the results of the sequences that they do not touch are right."""
    w = World("int8", 4, 2, 64, [300, 300, 300, 300], seed=36)
    settle(w, [300, 290, 280, 300])
    P = w.P
    b, start = w.batch([2, 1, 3, 1], advance=False)
    q = w.rows(7, 4, 1.5)
    plain = P.kv_attention(q, w.c, b)
    for groups in ([3, 1, 0], [-5, 2, 9], [2, 2, 2], [0, 4, 2], [2 ** 31 - 1, -2 ** 31, 7]):
        out = P.kv_attention_shared(q, w.c, b, dev([-3, 0]), group_start=dev(groups))
        torch.cuda.synchronize()
        err = (out.float() - plain.float()).abs().max().item()
        assert err <= 2 * 2.0 ** -8 * plain.float().abs().max().item()
        P.kv_attention_shared(q, w.c, b, dev([2, 2 ** 31 - 1]), group_start=dev(groups))
        torch.cuda.synchronize()


def test_unlike_value_scales_and_large_scores():
    w = World("int8", 8, 1, 128, [2000, 2000], seed=37)
    settle(w, [2000, 1990])
    share(w, [0, 2], [29])
    w.o.vs *= np.exp2(w.rng.integers(-90, 90, w.o.vs.shape)).astype(np.float32)
    w.c.v_scale.copy_(torch.from_numpy(w.o.vs))
    attend(w, [4, 1], [29])
    w.o.ks *= np.float32(64.0)
    w.c.k_scale.copy_(torch.from_numpy(w.o.ks))
    attend(w, [4, 1], [29])
    w.o.vs[w.table[0, :29]] = 0                          # a prefix of zeros, and one far above the rest
    w.c.v_scale.copy_(torch.from_numpy(w.o.vs))
    attend(w, [4, 1], [29])


@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_long_prefix_in_many_pieces(kind):
    w = World(kind, 8, 2, 64, [64 * 260, 64 * 4, 64 * 4], seed=38, extra=0)
    # one long table, the others' tables as wide: their own pages behind the prefix
    own = w.table[1:, :4].copy()
    w.table[1:, 254:258] = own
    w.table[1:, :254] = -1
    w.ctx[:] = [64 * 260 - 5, 64 * 256 + 7, 64 * 258]
    w.o.ks[:], w.o.vs[:] = 0.002, 0.01
    w.c.k_scale.fill_(0.002), w.c.v_scale.fill_(0.01)
    attend(w, [1, 1, 1], [254])
    attend(w, [6, 10, 20], [254])


def test_same_result_twice_and_workspace_of_any_content():
    w = World("int8", 8, 2, 128, [3000] * 6, seed=39)
    settle(w, [3000, 2800, 2900, 2600, 2990, 2570])
    share(w, [0, 6], [40])
    b, start = w.batch([1] * 6, advance=False)
    q = w.rows(6, 8, 1.5)
    ws = w.P.alloc_kv_shared_workspace(w.c, b, 8)
    got = []
    for fill in (0, 0xff, 0x5a):
        ws.fill_(fill)
        got += [w.P.kv_attention_shared(q, w.c, b, dev([40]), workspace=ws) for _ in range(3)]
    assert all(torch.equal(g, got[0]) for g in got)


def test_rows_outside_every_sequence_with_any_workspace():
    """Rows before the first and behind the last sequence, whose places in the workspace nobody writes."""
    w = World("int8", 4, 2, 64, [700, 500, 449], seed=42)
    settle(w, [700, 500, 449])
    share(w, [0, 3], [6])
    P = w.P
    b = P.KVBatch(torch.from_numpy(w.ctx.copy()).cuda(), torch.from_numpy(w.table).cuda(), dev([5, 6, 9, 10]), n_tokens=40, max_q=3)
    q = w.rows(40, 4, 1.5)
    ws = P.alloc_kv_shared_workspace(w.c, b, 4)
    got = []
    for fill in (0, 0x7f, 0xff):
        ws.fill_(fill)
        out = torch.full_like(q, 7.0)
        P.kv_attention_shared(q, w.c, b, dev([6]), out=out, workspace=ws)
        got.append(out)
    torch.cuda.synchronize()
    want, tol = OO.attention_shared(w.o, w.table, w.ctx, [5, 6, 9, 10], 3, f64(q), [6], None, 64 ** -0.5)
    for out in got:
        out = f64(out)
        assert (np.abs(out[5:10] - want[5:10]) <= tol[5:10]).all()
        assert (out[:5] == 7).all() and (out[10:] == 7).all()


def test_two_captured_graphs_share_a_workspace_as_lengths_move():
    w = World("fp8", 8, 2, 64, [900] * 4, seed=40)
    settle(w, [700, 600, 650, 580])
    share(w, [0, 4], [9])
    P = w.P
    ctx, table = torch.from_numpy(w.ctx.copy()).cuda(), torch.from_numpy(w.table).cuda()
    b = P.KVBatch(ctx, table)
    q, k, v = w.rows(4, 8, 1.5), w.rows(4, 2), w.rows(4, 2)
    ws = P.alloc_kv_shared_workspace(w.c, b, 8)
    sh = dev([9])
    graphs, outs = [], []
    for grow in (1, 0):
        out = torch.empty_like(q)

        def step():
            if grow:
                ctx.add_(1)
                P.kv_append(w.c, b, k, v)
            P.kv_attention_shared(q, w.c, b, sh, out=out, workspace=ws)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        graphs.append(g)
        outs.append(out)
    for i in range(12):
        q.copy_(w.rows(4, 8, 1.5))
        sh.fill_(9 - i % 3)                              # shared entries are read from the first sequence alone
        if i % 3:
            table[:, 9 - i % 3:9] = table[:1, 9 - i % 3:9]
        graphs[0].replay()
        graphs[1].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0], outs[1]), i
        assert torch.equal(outs[0], P.kv_attention_shared(q, w.c, b, sh)), i
        full = table.clone()
        full[1:, :9] = full[0, :9]
        near = P.kv_attention(q, w.c, P.KVBatch(ctx, full)).float()
        assert (outs[0].float() - near).abs().max() <= 2.0 ** -6 * near.abs().max()


def test_memory_let_go_before_the_stream_runs():
    w = World("int8", 8, 2, 128, [900, 700, 700], seed=41)
    settle(w, [900, 700, 690])
    share(w, [0, 3], [9])
    P = w.P
    b, start = w.batch([2, 1, 4], advance=False)
    q = w.rows(7, 8, 1.5)
    want = P.kv_attention_shared(q, w.c, b, dev([9]), group_start=dev([0, 3]))
    side = torch.cuda.Stream()
    sh0, gs0 = dev([9]), dev([0, 3])
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(400_000_000)      # the calls below wait behind this

    def calls():
        batch = P.KVBatch(b.ctx_len.clone(), b.block_table.clone(), b.q_start.clone(), n_tokens=7, max_q=4)
        qq, sh, gs = q.clone(), sh0.clone(), gs0.clone()
        side.wait_stream(torch.cuda.current_stream())
        out = P.kv_attention_shared(qq, w.c, batch, sh, group_start=gs, stream=side)
        return out, {t.data_ptr() for t in (qq, sh, gs, batch.ctx_len, batch.block_table, batch.q_start)}, \
            [t.nbytes for t in (qq, sh, gs, batch.block_table)]
    out, kept, sizes = calls()
    assert not side.query()
    junk = [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for n in sizes + [8, 12, 16] for _ in range(2)]
    again = {t.data_ptr() for t in junk}
    assert not side.query() and not kept & again
    torch.cuda.synchronize()
    assert torch.equal(out, want)


def test_nan_codes_that_a_shared_page_holds():
    """Every slot of a shared page holds a token, so a NaN among its values is one, as in the attention over all
    pages; one in the slots behind a sequence's last token is not."""
    w = World("fp8", 4, 2, 64, [300, 300, 290, 200], seed=41)
    settle(w, [300, 300, 290, 200])
    share(w, [0, 3, 4], [3, 1])
    q = [w.rows(n, 4, 1.5) for n in (4, 67)]
    new = ([1, 1, 1, 1], [5, 60, 1, 1])
    good = [attend(w, n, [3, 1], [0, 3, 4], q=x.clone()) for n, x in zip(new, q)]
    codes = w.c.v.view(w.o.n_pages, 2, -1)
    for s, pg, slot, head, ch in ((0, 1, 9, 1, 5), (0, 2, 63, 0, 60), (3, 0, 0, 0, 17), (3, 2, 4, 0, 3), (3, 3, 30, 1, 9), (1, 4, 50, 0, 8)):
        codes[int(w.table[s, pg]), head, ((ch // 16 * 4 + slot // 4 % 4) * 16 + ch % 16) * 16 + slot // 16 * 4 + slot % 4] = 0x7f
    for n, x, a in zip(new, q, good):
        b, start = w.batch(n, advance=False)
        out = w.P.kv_attention_shared(x, w.c, b, dev([3, 1]), group_start=dev([0, 3, 4]))
        nan = torch.zeros(x.shape, dtype=torch.bool)               # query heads 0, 1 read key head 0, heads 2, 3 the other
        nan[:start[3], 2:, 5] = nan[:start[3], :2, 60] = nan[start[3]:, :2, 17] = nan[start[3]:, :2, 3] = True
        assert torch.equal(out.isnan().cpu(), nan) and torch.equal(out.cpu()[~nan], a.cpu()[~nan])
