"""The operators around the paged cache without a GPU: refusals of the C ABI
(before anything is enqueued), the Python handles' checks, and pins of their oracle."""

import ctypes

import numpy as np
import pytest
import torch

import free_ffn_activation_prox_amd as P
from free_ffn_activation_prox_amd import _KVPool, _lib
from oracle import kv_oracle as KO
from oracle import kv_ops_oracle as OO
from test_kv_host import FAKE, INVALID, MISMATCH, UNSUPPORTED, WORKSPACE, batch, cache


def pool(**over):
    p = _KVPool(100, 4, 8, FAKE, FAKE, FAKE)
    for k, v in over.items():
        setattr(p, k, v)
    return p


def pages(p=None, want=FAKE, parent=None, shared=None, qs=FAKE, rows=10, slots=FAKE, status=FAKE, ws=FAKE, n=1 << 40):
    return _lib.prox_kv_pages(ctypes.byref(p or pool()), want, parent, shared, qs, rows, slots, status, ws, n, None)


def bounds(c=None, b=None, out=FAKE):
    return _lib.prox_kv_page_bounds(ctypes.byref(c or cache()), ctypes.byref(b or batch()), out, None)


def select(c=None, b=None, q=FAKE, qs=512, H=4, bnd=FAKE, keep=4, first=1, last=1, out=FAKE, ws=FAKE, n=1 << 40):
    return _lib.prox_kv_select(ctypes.byref(c or cache()), ctypes.byref(b or batch()), q, qs, H, bnd, keep, first, last,
                               out, ws, n, None)


def selected(c=None, b=None, q=FAKE, qs=512, H=4, lst=FAKE, keep=4, scale=0.1, out=2 * FAKE, os=512, ws=FAKE, n=1 << 40):
    return _lib.prox_kv_attention_selected(ctypes.byref(c or cache()), ctypes.byref(b or batch()), q, qs, H, lst, keep,
                                           scale, out, os, ws, n, None)


def shared(c=None, b=None, gs=FAKE, n=2, sh=FAKE, q=FAKE, qs=512, H=4, scale=0.1, out=2 * FAKE, os=512, ws=FAKE, bytes=1 << 40):
    return _lib.prox_kv_attention_shared(ctypes.byref(c or cache()), ctypes.byref(b or batch()), gs, n, sh, q, qs, H, scale,
                                         out, os, ws, bytes, None)


def test_pool_refusals():
    for over, want in ((dict(n_pages=0), INVALID), (dict(n_seq=0), INVALID), (dict(max_pages=0), INVALID),
                       (dict(n_pages=(1 << 24) + 1), UNSUPPORTED), (dict(n_seq=(1 << 24) + 1), UNSUPPORTED),
                       (dict(max_pages=1 << 26), UNSUPPORTED), (dict(refs=0), INVALID), (dict(ctx_len=0), INVALID),
                       (dict(block_table=0), INVALID), (dict(refs=FAKE + 2), INVALID), (dict(ctx_len=FAKE + 1), INVALID)):
        assert pages(p=pool(**over)) == want, over
        assert _lib.prox_kv_pages_workspace_bytes(ctypes.byref(pool(**over))) == 0
    for over in (dict(want=0), dict(qs=0), dict(status=0), dict(slots=0), dict(ws=0), dict(parent=FAKE), dict(shared=FAKE),
                 dict(rows=-1), dict(want=FAKE + 2), dict(ws=FAKE + 4), dict(slots=FAKE + 1)):
        assert pages(**over) == INVALID, over
    need = _lib.prox_kv_pages_workspace_bytes(ctypes.byref(pool()))
    assert need > 0 and pages(n=need - 1) == WORKSPACE


@pytest.mark.parametrize("call", [bounds, select, selected, shared])
def test_cache_and_batch_refusals(call):
    for over, want in ((dict(kind=0), INVALID), (dict(n_pages=0), INVALID), (dict(n_kv=1025), UNSUPPORTED),
                       (dict(head_dim=132), INVALID), (dict(head_pad=64), MISMATCH), (dict(k=0), INVALID)):
        assert call(c=cache(**over)) == want, over
    for over, want in ((dict(n_seq=0), INVALID), (dict(n_tokens=-1), INVALID), (dict(max_pages=0), INVALID),
                       (dict(max_pages=1 << 26), UNSUPPORTED), (dict(ctx_len=0), INVALID), (dict(q_start=0), INVALID)):
        assert call(b=batch(**over)) == want, over
    for b in (batch(n_tokens=0), batch(max_q=0)):
        assert call(b=b) == 0


def test_bounds_and_select_refusals():
    assert bounds(out=0) == INVALID and bounds(out=FAKE + 8) == INVALID
    assert select(q=0) == INVALID and select(bnd=0) == INVALID and select(out=0) == INVALID
    assert select(bnd=FAKE + 8) == INVALID and select(out=FAKE + 2) == INVALID
    assert select(H=5) == INVALID and select(H=1026) == UNSUPPORTED and select(qs=511) == INVALID
    assert select(keep=0, first=0) == INVALID and select(keep=(1 << 20) + 1) == UNSUPPORTED
    assert select(first=-1) == INVALID and select(last=0) == INVALID and select(keep=4, first=3, last=2) == INVALID
    assert select(first=0x7fffffff, last=0x7fffffff) == INVALID
    assert select(b=batch(max_pages=32769)) == UNSUPPORTED
    assert select(ws=0) == INVALID and select(ws=FAKE + 16) == INVALID
    for b in (batch(), batch(max_pages=2000), batch(n_seq=1, n_tokens=1, max_q=1, max_pages=32768)):
        need = _lib.prox_kv_select_workspace_bytes(ctypes.byref(cache()), ctypes.byref(b), 4)
        assert need > 0 and select(b=b, n=need - 1) == WORKSPACE
    assert _lib.prox_kv_select_workspace_bytes(ctypes.byref(cache()), ctypes.byref(batch(max_pages=32769)), 4) == 0


def test_selected_refusals():
    assert selected(q=0) == INVALID and selected(out=0) == INVALID and selected(out=FAKE) == INVALID
    assert selected(H=5) == INVALID and selected(H=1026) == UNSUPPORTED
    assert selected(qs=511) == INVALID and selected(os=500) == INVALID
    assert selected(lst=0) == INVALID and selected(lst=FAKE + 2) == INVALID
    assert selected(keep=0) == INVALID and selected(keep=(1 << 20) + 1) == UNSUPPORTED
    assert selected(scale=float("inf")) == INVALID and selected(scale=float("nan")) == INVALID
    assert selected(ws=0) == INVALID and selected(ws=FAKE + 16) == INVALID
    for keep in (1, 64, 5000):
        b = batch()
        need = _lib.prox_kv_selected_workspace_bytes(ctypes.byref(cache()), ctypes.byref(b), 4, keep)
        assert need > 0 and selected(keep=keep, n=need - 1) == WORKSPACE
    big = batch(n_tokens=1 << 28, max_q=1 << 28)
    c = cache(n_kv=64)
    assert _lib.prox_kv_selected_workspace_bytes(ctypes.byref(c), ctypes.byref(big), 64, 4) == 0
    assert selected(c=c, b=big, H=64, qs=64 * 128, os=64 * 128) == UNSUPPORTED


def test_shared_refusals():
    assert shared(q=0) == INVALID and shared(out=0) == INVALID and shared(out=FAKE) == INVALID
    assert shared(H=5) == INVALID and shared(H=1026) == UNSUPPORTED
    assert shared(qs=511) == INVALID and shared(os=500) == INVALID
    assert shared(n=0) == INVALID and shared(n=4) == INVALID and shared(gs=0) == INVALID
    assert shared(sh=0) == INVALID and shared(sh=FAKE + 2) == INVALID and shared(gs=FAKE + 1) == INVALID
    assert shared(scale=float("inf")) == INVALID and shared(scale=float("nan")) == INVALID
    assert shared(ws=0) == INVALID and shared(ws=FAKE + 16) == INVALID
    need = _lib.prox_kv_shared_workspace_bytes(ctypes.byref(cache()), ctypes.byref(batch()), 4, 2)
    assert need > 0 and shared(bytes=need - 1) == WORKSPACE
    assert shared(gs=0, n=1, bytes=0) == WORKSPACE
    for over in (dict(n_seq=1 << 20, n_tokens=1 << 20, max_q=1, max_pages=300),
                 dict(n_seq=1 << 28, n_tokens=1 << 28, max_q=1 << 28, max_pages=(1 << 25) - 1)):
        b, c = batch(**over), cache(n_kv=8)
        assert _lib.prox_kv_shared_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 32, 1) == 0
        assert shared(c=c, b=b, H=32, qs=32 * 128, os=32 * 128, n=1) == UNSUPPORTED


def test_python_handles_refuse_host_tensors_and_shapes():
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        P.KVPool(torch.zeros(9, dtype=torch.int32), i, torch.zeros(3, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        P.KVPool(torch.zeros(9, dtype=torch.int32), i, torch.zeros(2, 4, dtype=torch.int32))


def test_oracle_pool_conserves_pages():
    r = np.random.default_rng(1)
    o = OO.Pool(60, 7, 12)
    for _ in range(60):
        want = np.where(r.random(7) < 0.2, 0, np.maximum(o.ctx + r.integers(-90, 120, 7), 0))
        q_start, slots, status = o.move(want, 2000, r.integers(-1, 7, 7), r.integers(0, 5, 7))
        # each page's count is how often the tables name it; the rest of a row is -1
        names = o.table[o.table >= 0]
        assert np.array_equal(np.bincount(names, minlength=60), o.refs)
        assert np.array_equal((o.table >= 0).sum(1), -(-o.ctx // 64))
        assert status[1] == (o.refs == 0).sum()
        used = slots[:q_start[-1]]
        assert (used >= 0).all() and np.unique(used).size == used.size and (slots[q_start[-1]:] == -1).all()
        assert (o.refs[used // 64] == 1).all()                       # nothing new goes into a shared page


def test_oracle_bounds_hold_for_every_query():
    r = np.random.default_rng(2)
    for kind in ("int8", "fp8"):
        c = KO.Cache(kind, 3, 2, 24)
        c.k = r.integers(0, 256, c.k.shape).astype(np.uint8)
        table = np.array([[2, 0]], np.int32)
        b = np.zeros((3, 2, 2, c.hp), np.int8)
        OO.bounds(c, table, [100], None, 1, 1, b)                     # one token: the page that it lies in
        assert not b[1].any() and not b[2].any()
        OO.bounds(c, table, [100], np.array([0, 100]), 100, 100, b)
        tok = np.nan_to_num(KO.decode(kind, c.tokens("k")), nan=0.0) * (1.0 if kind == "int8" else 127 / 448)
        for pg, held in ((2, 64), (0, 36)):
            for _ in range(20):
                q = r.standard_normal((2, c.hp))
                top = np.maximum(q * b[pg, :, 0], q * b[pg, :, 1]).sum(-1)
                assert ((tok[pg, :, :held] * q[:, None]).sum(-1).max(-1) <= top + 1e-9).all()


def test_more_threads_than_a_launch_has_are_refused_before_the_first():
    """2^32 threads: what is one short of them has a workspace, what reaches them has none and is refused."""
    def both(size, call, c, over, fits):
        b = batch(**over)
        assert (size(c, b) > 0) == fits, over
        if not fits:
            assert call(c, b) == UNSUPPORTED, over

    one = lambda n: dict(n_seq=n, n_tokens=n, max_q=1, q_start=0)                                     # noqa: E731
    size = lambda c, b: _lib.prox_kv_select_workspace_bytes(ctypes.byref(c), ctypes.byref(b), c.n_kv)  # noqa: E731
    call = lambda c, b: select(c=c, b=b, H=c.n_kv, qs=c.n_kv * 128, n=(1 << 62))                       # noqa: E731
    both(size, call, cache(n_kv=1), one((1 << 24) - 1), True)                                         # a block of 256 a row
    both(size, call, cache(n_kv=1), one(1 << 24), False)
    both(size, call, cache(n_kv=8), one(1 << 21), False)
    size = lambda c, b: _lib.prox_kv_selected_workspace_bytes(ctypes.byref(c), ctypes.byref(b), c.n_kv, 4)  # noqa: E731
    call = lambda c, b: selected(c=c, b=b, H=c.n_kv, qs=c.n_kv * 128, os=c.n_kv * 128, n=(1 << 62))         # noqa: E731
    both(size, call, cache(n_kv=1), one((1 << 24) - 1), True)
    both(size, call, cache(n_kv=1), one(1 << 24), False)
    both(size, call, cache(n_kv=8), one(1 << 21), False)
    # the join of a shared prefix: head_pad / 4 threads a row and query head
    size = lambda c, b: _lib.prox_kv_shared_workspace_bytes(ctypes.byref(c), ctypes.byref(b), 64, 1)        # noqa: E731
    call = lambda c, b: shared(c=c, b=b, n=1, H=64, qs=64 * 128, os=64 * 128, bytes=1 << 62)                # noqa: E731
    for n, fits in (((1 << 21) - 4, True), (1 << 21, False), (1 << 24, False)):
        both(size, call, cache(n_kv=8), dict(n_seq=n // 64, n_tokens=n, max_q=64), fits)
