"""Page tables on the GPU (kv_pages) against the oracle's sequential form:
every array of the pool, rows, slots and status, whole numbers."""

import numpy as np
import pytest
import torch

from oracle import kv_ops_oracle as OO

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def dev(a):
    return torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


class Pair:
    """The same pool on the GPU and in the oracle."""

    def __init__(self, n_pages, n_seq, max_pages):
        import free_ffn_activation_prox_amd as P
        self.P = P
        self.p = P.KVPool.alloc(n_pages, n_seq, max_pages)
        self.o = OO.Pool(n_pages, n_seq, max_pages)

    def move(self, want, n_rows=None, parent=None, shared=None, **kw):
        want = np.asarray(want, np.int32)
        if n_rows is None:
            n_rows = int(np.maximum(want, 0).sum()) + 5
        got = self.P.kv_pages(self.p, dev(want), n_rows, parent=None if parent is None else dev(parent),
                              shared=None if shared is None else dev(shared), **kw)
        torch.cuda.synchronize()
        exp = self.o.move(want, n_rows, parent, shared)
        for n, a, b in zip(("q_start", "slots", "status"), got, exp):
            assert np.array_equal(a.cpu().numpy(), b), n
        self.same()
        return exp

    def same(self):
        for n, a, b in (("ctx", self.p.ctx_len, self.o.ctx), ("table", self.p.block_table, self.o.table),
                        ("refs", self.p.refs, self.o.refs)):
            assert np.array_equal(a.cpu().numpy(), b), n


def test_grow_cut_back_and_end():
    w = Pair(40, 5, 12)
    w.move([1, 64, 65, 0, 700])
    w.move([2, 65, 60, 1, 700])          # one page more, one less
    w.move([64, 65, 0, 300, 5])          # ends; a long one is cut back
    w.move([64, 65, 128, 300, 768])      # freed pages are taken again, lowest first
    w.move([0, 0, 0, 0, 0])
    assert (w.o.refs == 0).all()


def test_pool_runs_out_and_table_is_too_short():
    w = Pair(10, 4, 8)
    assert w.move([300, 300, 64, 1])[2].tolist() == [2, 0]         # 5 + 5 pages; the others are refused
    assert w.move([300, 128, 64, 1])[2].tolist() == [0, 1]         # what one gives back the next ones get
    assert w.move([300, 128, 600, 65])[2].tolist() == [1, 0]       # 10 pages exceed a row of the table
    assert w.move([2147483647, 128, -5, 65], n_rows=99)[2][0] == 1


def test_a_refused_sequence_refuses_later_ones_that_need_pages_only():
    w = Pair(6, 4, 8)
    w.move([64, 60, 64, 60])
    st = w.move([64 * 4, 61, 65, 62])[2]                           # 3 of 2 free pages; 1 of them after it
    assert st.tolist() == [2, 2]


def test_begin_with_the_pages_of_another():
    w = Pair(64, 6, 16)
    w.move([500, 0, 0, 0, 30, 0])
    par, sh = [-1, 0, 0, 0, 0, 4], [0, 7, 3, 100, 7, 1]
    w.move([520, 448, 200, 460, 31, 70], parent=par, shared=sh)    # whole pages only: 7, 3, 7; 4 has tokens; 5's parent no whole page
    w.move([0, 449, 201, 461, 32, 0], parent=[-1] * 6, shared=[0] * 6)   # the parent ends, its pages stay
    w.move([64, 0, 0, 0, 0, 0])
    assert w.o.refs.sum() == 1


def test_parent_that_ends_or_is_cut_in_the_same_call():
    w = Pair(64, 4, 16)
    w.move([400, 300, 0, 0])
    w.move([0, 10, 400, 300], parent=[-1, -1, 0, 1], shared=[0, 0, 6, 4])
    w.move([100, 10, 64, 300], parent=[2, -1, -1, -1], shared=[1, 0, 0, 0])
    assert w.o.refs.max() == 2


def test_child_shorter_than_what_it_takes_and_parents_out_of_range():
    w = Pair(32, 5, 8)
    w.move([512, 0, 0, 0, 0])
    w.move([512, 100, 0, 5, 70], parent=[0, 0, 0, 9, -3], shared=[2, 8, 8, 8, 8])
    w.move([512, 164, 1, 5, 70], parent=[0, 0, 2, 3, 4], shared=[-2] * 5)


def test_going_on_in_a_shared_page_is_refused():
    w = Pair(32, 3, 8)
    w.move([256, 0, 0])
    w.move([256, 256, 0], parent=[-1, 0, -1], shared=[0, 4, 0])
    w.move([256, 100, 0])                                          # cut back into a page that sequence 0 holds too
    assert w.move([256, 101, 0])[2].tolist()[0] == 1
    w.move([0, 100, 0])                                            # now it is alone
    assert w.move([0, 101, 0])[2].tolist()[0] == 0


def test_rows_that_do_not_fit():
    w = Pair(32, 3, 8)
    for n in (0, 1, 100, 129):
        w.move([100, 30, 0], n_rows=n)
        w.move([0, 0, 0])


# the last ones in several blocks: many pages, many sequences, long tables
@pytest.mark.parametrize("n_pages,n_seq,max_pages,top", [(1, 1, 1, 70), (3000, 1100, 9, 500), (5000, 70, 200, 9000),
                                                         (129, 17, 40, 2000), (70003, 300, 300, 19000), (2047, 1024, 3, 190),
                                                         (33000, 5000, 12, 700), (66000, 3, 30000, 1900000)])
def test_random_steps(n_pages, n_seq, max_pages, top):
    w = Pair(n_pages, n_seq, max_pages)
    r = np.random.default_rng(n_pages)
    for step in range(5):
        want = np.where(r.random(n_seq) < 0.2, 0, w.o.ctx + r.integers(-70, 140, n_seq))
        want = np.where(r.random(n_seq) < 0.3, r.integers(0, top, n_seq), want)
        par = r.integers(-1, n_seq, n_seq)
        w.move(want, parent=par, shared=r.integers(0, 6, n_seq))
        # steps of a token or two, and back, in one block; more rows than that call says, too
        for _ in range(3):
            w.move(w.o.ctx + r.integers(-2, 3, n_seq), n_rows=2 * n_seq)
        w.move(np.where(r.random(n_seq) < 0.4, 0, w.o.ctx + r.integers(0, 90, n_seq)), n_rows=n_seq)


@pytest.mark.parametrize("n_pages,max_pages", [(200, 16), (70000, 16)])
def test_captured_and_replayed(n_pages, max_pages):
    import free_ffn_activation_prox_amd as P
    w = Pair(n_pages, 8, max_pages)
    want, par, sh = (torch.zeros(8, dtype=torch.int32, device="cuda") for _ in range(3))
    par.fill_(-1)
    r = np.random.default_rng(5)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        P.kv_pages(w.p, want, 300, parent=par, shared=sh)
    torch.cuda.current_stream().wait_stream(side)
    w.o.move([0] * 8, 300)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = P.kv_pages(w.p, want, 300, parent=par, shared=sh)
    for k in range(6):
        nw = np.where(w.o.ctx == 0, r.integers(0, 600, 8), w.o.ctx + r.integers(0, 70, 8)) * (r.random(8) > 0.2)
        want.copy_(dev(nw))
        par.copy_(dev([-1, 0, 0, 1, 1, 2, -1, 3]))
        sh.fill_(k)
        g.replay()
        exp = w.o.move(nw, 300, [-1, 0, 0, 1, 1, 2, -1, 3], [k] * 8)
        torch.cuda.synchronize()
        assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, exp)), k
        w.same()
        torch.ones(1000, device="cuda").sum().item()               # eager work between the replays


def test_arrays_at_any_four_bytes():
    import free_ffn_activation_prox_amd as P
    w = Pair(301, 5, 9)
    odd = lambda n, v: torch.full((n + 3,), v, dtype=torch.int32, device="cuda")[3:]  # noqa: E731
    w.p = P.KVPool(odd(301, 0), odd(5, 0), odd(45, -1).view(5, 9))
    w.move([70, 500, 0, 64, 1], q_start=odd(6, 9), slots=odd(640, 9), status=odd(2, 9), n_rows=640)
    w.move([71, 0, 128, 64, 2], n_rows=10)


def test_pool_feeds_append_and_attention():
    """A run of calls as a server makes them: the pool's arrays as a batch's."""
    from oracle import kv_oracle as KO
    from test_gpu_kv import World, f64
    w = World("int8", 4, 2, 64, [300, 300, 300], seed=9, extra=0)
    P = w.P
    pool = P.KVPool.alloc(w.o.n_pages, 3, w.table.shape[1])
    for want in ([100, 0, 70], [101, 200, 0], [164, 260, 90]):
        T = 400
        q_start, slots, status = P.kv_pages(pool, dev(want), T)
        assert status.tolist()[0] == 0
        b = P.KVBatch(pool.ctx_len, pool.block_table, q_start, n_tokens=T, max_q=T)
        k, v, q = w.rows(T, 2), w.rows(T, 2), w.rows(T, 4, 1.5)
        P.kv_append(w.c, b, k, v)
        w.ctx, w.table, start = pool.ctx_len.cpu().numpy(), pool.block_table.cpu().numpy(), q_start.cpu().numpy()
        KO.append(w.o, w.table, w.ctx, start, T, f64(k), f64(v))
        w.same_cache()
        w.attend(b, start, q=q)
        # a row's slot is where its key went
        kt = KO.Cache.tokens(w.o, "k")
        for row in (0, int(start[-1]) - 1):
            slot = int(slots[row])
            got = KO.decode("int8", kt[slot // 64, 0, slot % 64, :64]) * w.o.ks[slot // 64, 0]
            assert np.abs(got - f64(k)[row, 0]).max() <= 0.51 * w.o.ks[slot // 64, 0] * 2
        assert (slots[int(start[-1]):] == -1).all()


def test_on_a_stream_of_its_own():
    import free_ffn_activation_prox_amd as P
    w = Pair(100, 4, 20)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
    want = dev([300, 10, 0, 64])
    side.wait_stream(torch.cuda.current_stream())
    got = P.kv_pages(w.p, want, 400, stream=side)
    del want
    junk = [torch.full((4,), 9, dtype=torch.int32, device="cuda") for _ in range(8)]
    exp = w.o.move([300, 10, 0, 64], 400)
    torch.cuda.synchronize()
    assert all(np.array_equal(a.cpu().numpy(), b) for a, b in zip(got, exp))
    w.same()
    del junk


def test_as_many_sequences_as_a_pool_may_have():
    """2^24 sequences (PROX_KV_MAX_POOL), a handful of which have tokens: the first, the last and some between."""
    import free_ffn_activation_prox_amd as P
    n = 1 << 24
    pool = P.KVPool.alloc(40, n, 2)
    at = torch.tensor([0, 5, 255, 256, 1 << 20, (1 << 20) + 1, n - 257, n - 1], device="cuda")
    for top, status in ((100, [0, 40 - 16]), (1, [0, 40 - 8]), (0, [0, 40])):
        want = torch.zeros(n, dtype=torch.int32, device="cuda")
        want[at] = torch.arange(8, dtype=torch.int32, device="cuda") + top if top else 0
        had = pool.ctx_len[at].clone()
        q_start, slots, st = P.kv_pages(pool, want, 900)
        torch.cuda.synchronize()
        assert st.tolist() == status and torch.equal(pool.ctx_len, want)
        pages = -(-want[at] // 64)
        rows = torch.clamp(want[at] - had, min=0)
        assert torch.equal(q_start[at + 1] - q_start[at], rows) and int(q_start[-1]) == int(rows.sum())
        assert torch.equal((pool.block_table[at] >= 0).sum(1), pages.long()) and int((pool.block_table >= 0).sum()) == int(pages.sum())
        assert int(pool.refs.sum()) == int(pages.sum()) and int(pool.refs.max()) <= 1
        assert int((slots >= 0).sum()) == int(rows.sum())
