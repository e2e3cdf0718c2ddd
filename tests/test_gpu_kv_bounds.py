"""GPU checks of the paged 8-bit cache where a batch's bounds say little about
the batch: wide tables, a max_q beyond the tokens, offsets that do not rise."""

import numpy as np
import pytest
import torch

from test_gpu_kv import World, settle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_long_chunk_beside_single_tokens_with_a_wide_table():
    # 17 tiles of 256 tokens in the longest of 300 sequences and a table of 110000 pages each: by
    # n_seq, max_q and max_pages alone more than 2^31 pages to see; in truth some thousand
    lens = [4300] + [1 + 7 * s % 200 for s in range(299)]
    w = World("int8", 4, 4, 64, lens, seed=83)
    P = w.P
    settle(w, lens)
    new = [4200] + [1] * 299
    b, start = w.batch(new, advance=False)
    q = w.rows(b.n_tokens, 4)
    want = P.kv_attention(q, w.c, b)
    wide = torch.full((300, 110000), -1, dtype=torch.int32, device="cuda")
    wide[:, :w.table.shape[1]] = b.block_table
    far = P.KVBatch(b.ctx_len, wide, b.q_start, n_tokens=b.n_tokens, max_q=4200)
    assert torch.equal(P.kv_attention(q, w.c, far), want)
    k, v = P.kv_read(w.c, b)
    for t, r in zip(P.kv_read(w.c, far), (k, v)):
        assert torch.equal(t, r)


def test_max_q_beyond_the_tokens():
    lens = [700, 90, 1]
    w = World("fp8", 8, 2, 128, lens, seed=89)
    P = w.P
    settle(w, lens)
    for new in ([1, 1, 1], [3, 2, 1], [300, 60, 1]):
        b, start = w.batch(new, advance=False)
        q = w.rows(b.n_tokens, 8)
        want, _ = w.attend(b, start, q=q)
        k, v = P.kv_read(w.c, b)
        for loose in (b.n_tokens, 5000, 1 << 28, 0x7fffffff):
            far = P.KVBatch(b.ctx_len, b.block_table, b.q_start, n_tokens=b.n_tokens, max_q=loose)
            got = P.kv_attention(q, w.c, far)
            # another max_q may choose other tiles, so other roundings: 2^-7 of a value is two steps of bfloat16
            assert torch.allclose(got.float(), want.float(), rtol=2.0 ** -7, atol=1e-3), (new, loose)
            assert all(torch.equal(a, r) for a, r in zip(P.kv_read(w.c, far), (k, v)))


def test_offsets_that_do_not_rise_stay_in_bounds():
    # every other sequence names all rows: more tiles than the bounds of a rising q_start
    n, S = 600, 100
    w = World("int8", 4, 2, 64, [n] * S, seed=97)
    P = w.P
    table = torch.from_numpy(np.repeat(w.table[:1], S, 0)).cuda()
    w.ctx[0] = n
    one = P.KVBatch(torch.tensor([n], dtype=torch.int32, device="cuda"), table[:1].contiguous(),
                    torch.tensor([0, n], dtype=torch.int32, device="cuda"), n_tokens=n)
    P.kv_append(w.c, one, w.rows(n, 2), w.rows(n, 2))
    q = w.rows(n + 5, 4)
    want = P.kv_attention(q[:n], w.c, one)
    start = torch.tensor([0, n] * (S // 2) + [0], dtype=torch.int32, device="cuda")
    ctx = torch.full((S,), n, dtype=torch.int32, device="cuda")
    out = torch.full_like(q, 7.0)
    P.kv_attention(q, w.c, P.KVBatch(ctx, table, start, n_tokens=n + 5, max_q=n), out=out)
    torch.cuda.synchronize()
    # the sequences that are worked on all say the same of a row
    assert torch.allclose(out[:n].float(), want.float(), rtol=2.0 ** -7, atol=1e-3) and bool((out[n:] == 7).all())
    assert torch.equal(P.kv_attention(q[:n], w.c, one), want)


def test_numbers_past_32_bits_are_refused():
    w = World("int8", 4, 2, 64, [64], seed=103)
    P = w.P
    b, _ = w.batch([4])
    q = w.rows(4, 4)
    for call in (lambda: P.KVBatch(b.ctx_len, b.block_table, b.q_start, n_tokens=4, max_q=1 << 32),
                 lambda: P.KVBatch(b.ctx_len, b.block_table, b.q_start, n_tokens=(1 << 32) + 4),
                 lambda: P.kv_attention(q, w.c, b, window=1 << 32), lambda: P.kv_attention(q, w.c, b, window=(1 << 32) + 2)):
        with pytest.raises(ValueError):
            call()
    assert torch.equal(P.kv_attention(q, w.c, b, window=0x7fffffff), P.kv_attention(q, w.c, b))


def test_one_row_of_any_stride():
    # a batch of one row: the distance to a next one says nothing
    w = World("fp8", 4, 2, 64, [80], seed=107)
    P = w.P
    settle(w, [79])
    ref, got = [], []
    x = w.rows(1, 8)
    codes = w.c.k.clone(), w.c.v.clone(), w.c.k_scale.clone(), w.c.v_scale.clone()
    for out, stride in ((ref, 512), (got, 515)):
        for t, was in zip((w.c.k, w.c.v, w.c.k_scale, w.c.v_scale), codes):
            t.copy_(was)
        wide = torch.zeros(2, stride, dtype=torch.bfloat16, device="cuda")
        wide[0, :512] = x.flatten()
        q, k, v = (wide.as_strided((1, n, 64), (stride, 64, 1), a) for a, n in ((0, 4), (256, 2), (384, 2)))
        batch = P.KVBatch(torch.tensor([80], dtype=torch.int32, device="cuda"), torch.from_numpy(w.table).cuda())
        out.append(P.kv_append(w.c, batch, k, v, rot=w.rot.cuda(), q=q).clone())
        out.append(P.kv_append(w.c, batch, k, v, rot=w.rot.cuda(), q=q.clone(), q_out=q).clone())
        into = torch.zeros(2, stride, dtype=torch.bfloat16, device="cuda").as_strided((1, 4, 64), (stride, 64, 1))
        out.append(P.kv_attention(q, w.c, batch, out=into))
        out += [w.c.k.clone(), w.c.v.clone()]
    assert all(torch.equal(a, b) for a, b in zip(ref, got))
