"""The decode harness over a pool of pages where the pool ends: replayed steps that
the host does not count, refusals, and captured steps that outlive a shared prefix.

What must not change is compared code by code; outputs go by the 2e-2 bound of the
dense harness's test, as two harnesses may cut a sequence's pages in other places."""

import pytest
import torch

from test_gpu_decode_kv import SHAPE, _rel, _x
from test_gpu_decode_ops import BOUND, _build

pytestmark = pytest.mark.gpu
D = SHAPE["d"]


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _capture(h, rows):
    """A captured step of rows that the caller sets in the returned buffer; it does not run here."""
    buf = torch.zeros(rows, D, device="cuda")
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = h.step(buf)
    return g, buf, out


def _replay(g, buf, out, x):
    buf.copy_(x)
    g.replay()
    torch.cuda.synchronize()
    return out.clone()


def _codes(h, pages=slice(None)):
    return [t[pages].clone() for kv in h.kv for t in (kv.k, kv.v, kv.k_scale, kv.v_scale)]


def _same(a, b):
    return all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("kw", [dict(), dict(keep_pages=3)])
def test_replays_past_the_pool_leave_refused_sequences_as_they_are(kw):
    h, twin = (_build(n_seq=2, n_pages=n, **kw) for n in (4, 30))
    for g in (h, twin):
        g.prefill(_x(62, D, 1), 0)
        g.prefill(_x(126, D, 2), 1)
    run = _capture(h, 2)
    for i in range(2):                                             # 64 and 128 tokens: three whole pages
        x = _x(2, D, 3 + i)
        a, b = _replay(*run, x), twin.step(x)
        assert _rel(a, b) <= BOUND
    assert h.ctx.tolist() == [64, 128]
    own = _codes(h, h.table[1, :2].long())
    for i in range(3):                                             # sequence 0 takes the fourth page, 1 is refused
        x = _x(2, D, 6 + i)
        a, b = _replay(*run, x), twin.step(x)
        assert _rel(a[0], b[0]) <= BOUND and torch.isfinite(a).all()
        assert h.ctx.tolist() == [65 + i, 128] and h.status.tolist() == [1, 0]
        assert _same(_codes(h, h.table[1, :2].long()), own)


@pytest.mark.parametrize("n_pages,max_ctx", [(2, 128), (9, 64)])
def test_a_refused_row_stores_nothing(n_pages, max_ctx):
    """Both sequences refused, for want of pages or of entries in the table: the step without a pool over a table
    that names no page there, or past max_ctx."""
    h, other = _build(n_seq=2, n_pages=n_pages, max_ctx=max_ctx), _build(n_seq=2, max_ctx=max_ctx)
    for g in (h, other):
        g.prefill(_x(63, D, 1), 0)
        g.prefill(_x(63, D, 2), 1)
    other.table[:, 1:] = -1
    a, b = _capture(h, 2), _capture(other, 2)
    x = _x(2, D, 3)
    assert torch.equal(_replay(*a, x), _replay(*b, x))
    own = _codes(h)
    for i in range(2):
        x = _x(2, D, 4 + i)
        other.ctx.fill_(64)                                        # without a pool a step goes on
        assert torch.equal(_replay(*a, x), _replay(*b, x))
        assert h.ctx.tolist() == [64, 64] and h.status.tolist() == [2, n_pages - 2] and _same(_codes(h), own)


@pytest.mark.parametrize("kw", [dict(), dict(keep_pages=3)])
def test_a_context_that_the_pool_cannot_hold_changes_nothing(kw):
    h, twin = (_build(n_seq=2, n_pages=5, **kw) for _ in range(2))
    for g in (h, twin):
        g.share_prefix(_x(130, D, 1))
    before, codes, space = (h.lengths[:], h.pos, h.prefix, h.ctx.tolist(), h.pool.refs.tolist()), _codes(h), h.kv_ws
    with pytest.raises(ValueError):
        h.fill_cache(200)                                          # 8 pages
    assert before == (h.lengths[:], h.pos, h.prefix, h.ctx.tolist(), h.pool.refs.tolist())
    assert _same(_codes(h), codes) and h.kv_ws is space
    x = _x(2, D, 2)
    assert torch.equal(h.step(x), twin.step(x))
    with pytest.raises(ValueError):
        h.prefill(_x(190, D), 1)                                   # what the host counts is still there
    h.fill_cache(100)
    assert h.ctx.tolist() == [100, 100] and h.lengths == [100, 100]


def test_a_step_captured_before_a_prefix_goes_on_beside_it():
    """It reads every sequence's own table; the step that the harness now makes reads the prefix once.
    Neither uses memory that the harness has let go of."""
    h, twin = (_build(n_seq=3, n_pages=24) for _ in range(2))
    run = _capture(h, 3)
    spaces = [t.data_ptr() for t in (h.kv_ws, h.share_ws, h.shared)]
    h.fill_cache(0)                                                # the host counts the captured step: begin again
    for g in (h, twin):
        g.share_prefix(_x(64 * 3 + 5, D, 1))
    assert spaces == [t.data_ptr() for t in (h.kv_ws, h.share_ws, h.shared)]
    for i in range(3):
        x = _x(3, D, 2 + i)
        y = twin.step(x)
        assert _rel(_replay(*run, x), y) <= BOUND
        junk = torch.full((1 << 20,), float("nan"), device="cuda")  # takes the memory that is free
        assert h.ctx.tolist() == twin.ctx.tolist()
        del junk


def test_a_step_captured_with_a_prefix_goes_on_without_one():
    h, twin = (_build(n_seq=3, n_pages=24) for _ in range(2))
    h.share_prefix(_x(64 * 3 + 5, D, 1))
    run = _capture(h, 3)
    spaces = [t.data_ptr() for t in (h.kv_ws, h.share_ws, h.shared)]
    for g in (h, twin):
        g.fill_cache(300, seed=4)                                  # each sequence has pages of its own again
    assert spaces == [t.data_ptr() for t in (h.kv_ws, h.share_ws, h.shared)]
    for i in range(3):
        x = _x(3, D, 2 + i)
        y = twin.step(x)
        assert _rel(_replay(*run, x), y) <= BOUND
    assert h.ctx.tolist() == twin.ctx.tolist() == [303] * 3


def test_replays_past_the_pool_leave_a_shared_page_as_it_is():
    """Sequences that end where the prefix does, and one page for three of them."""
    h = _build(n_seq=3, n_pages=3)
    run = _capture(h, 3)
    h.fill_cache(0)
    h.share_prefix(_x(128, D, 1))
    prompt = _codes(h, h.table[0, :2].long())
    for i in range(3):
        y = _replay(*run, _x(3, D, 2 + i))
        assert torch.isfinite(y).all() and h.ctx.tolist() == [129 + i, 128, 128] and h.status.tolist() == [2, 0]
        assert _same(_codes(h, h.table[0, :2].long()), prompt)


def test_a_prompt_behind_replayed_steps_counts_them():
    """Replays move the lengths on the device alone: a prompt, a prefix or the pool's end is judged by those."""
    h = _build(n_seq=2, n_pages=4)
    h.prefill(_x(62, D, 1), 0)
    h.prefill(_x(126, D, 2), 1)
    run = _capture(h, 2)
    for i in range(4):                                             # 66 tokens in two pages, 128 in two
        _replay(*run, _x(2, D, 3 + i))
    assert h.ctx.tolist() == [66, 128]
    codes = _codes(h)
    with pytest.raises(ValueError):
        h.prefill(_x(1, D, 9), 1)                                  # a third page: the host had counted 127 tokens
    assert h.ctx.tolist() == h.lengths == [66, 128] and h.pos == 128 and _same(_codes(h), codes)
    assert torch.isfinite(h.prefill(_x(62, D, 9), 0)).all()        # its second page's last tokens
    with pytest.raises(ValueError):
        h.prefill(_x(1, D, 9), 0)
    h.fill_cache(0)
    _replay(*run, _x(2, D, 8))
    with pytest.raises(ValueError):
        h.share_prefix(_x(70, D))                                  # a token each
    assert h.ctx.tolist() == h.lengths == [1, 1]


def test_a_captured_prompt_that_the_pool_refuses():
    """Its rows have no position, as those of a step; past it, a prompt that fits goes on."""
    h, twin = (_build(n_seq=2, n_pages=n) for n in (3, 30))
    buf = torch.zeros(70, D, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        h.prefill(buf, 0)
    torch.cuda.current_stream().wait_stream(side)
    h.fill_cache(0)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = h.prefill(buf, 1)
    x = _x(70, D, 1)
    assert _rel(_replay(g, buf, out, x), twin.prefill(x, 1)) <= BOUND
    codes = _codes(h)
    y = _replay(g, buf, out, x)                                    # 140 tokens: a third page, which is there
    assert _rel(y, twin.prefill(x, 1)) <= BOUND and h.ctx.tolist() == [0, 140]
    own = _codes(h)
    y = _replay(g, buf, out, x)
    assert torch.isfinite(y).all() and h.ctx.tolist() == [0, 140] and _same(_codes(h), own) and not _same(own, codes)
