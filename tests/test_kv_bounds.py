"""Bounds of a batch of the paged 8-bit cache (no GPU): what fits one call of the
attention and what is refused, before anything is enqueued."""

import ctypes

import pytest

from test_kv_host import UNSUPPORTED, WORKSPACE, _lib, attend, batch, cache


def ws(c, b, heads):
    return _lib.prox_kv_workspace_bytes(ctypes.byref(c), ctypes.byref(b), heads)


def both(b, heads=32, **c):
    """Workspace bytes, and what a call with too small a workspace says (it never launches)."""
    c = cache(n_kv=8, **c)
    return ws(c, b, heads), attend(c=c, b=b, H=heads, qs=heads * 128, os=heads * 128, n=0)


def test_a_long_chunk_beside_single_tokens_fits():
    # 256 sequences, one of them a 32768-token chunk: 4 query heads a key head, tiles of 64 tokens
    need, st = both(batch(n_seq=256, n_tokens=32768 + 255, max_q=32768, max_pages=2048))
    assert need > 0 and st == WORKSPACE


@pytest.mark.parametrize("over", [
    dict(n_seq=256, n_tokens=32768 * 256, max_q=32768, max_pages=2048),      # all of them so long
    dict(n_seq=1 << 20, n_tokens=1 << 20, max_q=1, max_pages=300),
    dict(n_seq=1 << 28, n_tokens=1 << 28, max_q=1 << 28, max_pages=(1 << 25) - 1),
    dict(n_seq=1 << 28, n_tokens=1 << 28, max_q=0x7fffffff, max_pages=(1 << 25) - 1),
])
def test_what_is_refused_has_no_workspace(over):
    assert both(batch(**over)) == (0, UNSUPPORTED)


def test_max_q_beyond_the_tokens_changes_nothing():
    for n in (1, 5, 400):
        for loose in (n, 1000, 1 << 28, 0x7fffffff):
            need, st = both(batch(n_seq=1, n_tokens=n, max_q=loose, max_pages=100))
            assert need > 0 and st == WORKSPACE, (n, loose)
    a, _ = both(batch(n_seq=3, n_tokens=10, max_q=0x7fffffff))
    assert a == both(batch(n_seq=3, n_tokens=10, max_q=1 << 28))[0]


def test_workspace_of_a_batch_serves_others_of_its_shape():
    # the same n_seq, max_q and max_pages, any number of tokens
    for heads in (8, 32, 72, 200, 1024):
        for dim in (64, 128, 256):
            for max_q in (1, 2, 3, 16, 17, 33, 300, 5000):
                for n_seq in (1, 3, 64):
                    for pages in (1, 40, 3000):
                        # a batch within the stated bound of tiles times pages is never refused
                        got = {ws(cache(n_kv=8, head_dim=dim, head_pad=dim),
                                  batch(n_seq=n_seq, n_tokens=n, max_q=max_q, max_pages=pages), heads)
                               for n in (0, 1, n_seq, max_q, max_q + n_seq, n_seq * max_q)
                               if (n * heads // 64 + n_seq * max(8, heads // 64)) * (pages + 3) < 1 << 31}
                        assert len(got) == 1 and 0 not in got, (heads, dim, max_q, n_seq, pages, got)


def test_line_leaves_room_for_a_piece():
    # 64 key heads: one unit for each page and one for the segment, 64 (max_pages + 1) in all.  A block adds
    # its piece, a 256th of the line without a GPU, to units of the line in 32 bits
    for pages, fits in ((33554430, False), (33554431 - (1 << 16), False), (33000000, True)):
        b = batch(n_seq=1, n_tokens=1, max_q=1, max_pages=pages)
        c = cache(n_kv=64)
        assert 64 * (pages + 1) < 1 << 31
        need, st = ws(c, b, 64), attend(c=c, b=b, H=64, qs=64 * 128, os=64 * 128, n=0)
        assert (need > 0, st) == ((True, WORKSPACE) if fits else (False, UNSUPPORTED)), pages
