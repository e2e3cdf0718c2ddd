"""The paged 8-bit cache's calls on a stream given with `stream`: what a caller
lets go of before the stream has run stays the call's."""

import pytest
import torch

from test_gpu_kv import World, settle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def test_memory_let_go_before_the_stream_runs():
    w = World("int8", 8, 2, 128, [700, 300], seed=101)
    P = w.P
    settle(w, [700, 300])
    b, start = w.batch([200, 90], advance=False)
    q, k, v = w.rows(290, 8), w.rows(290, 2), w.rows(290, 2)
    rot = w.rot.cuda()
    g = torch.ones(128, device="cuda")
    scales = w.c.k_scale.clone(), w.c.v_scale.clone()
    codes = w.c.k.clone(), w.c.v.clone()
    qr = P.kv_append(w.c, b, k, v, q=q, rot=rot, g_q=g, g_k=g)
    want = P.kv_attention(qr, w.c, b)
    kr, vr = P.kv_read(w.c, b)
    for t, was in zip((w.c.k, w.c.v, w.c.k_scale, w.c.v_scale), codes + scales):
        t.copy_(was)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(50_000_000)        # the calls below wait behind this
    # inputs, handles and workspace of the current stream, gone when the calls return
    def calls():
        batch = P.KVBatch(b.ctx_len.clone(), b.block_table.clone(), b.q_start.clone(), n_tokens=290, max_q=200)
        ins = [t.clone() for t in (q, k, v, rot, g, g)]
        into = torch.empty_like(q)
        ws = P.alloc_kv_workspace(w.c, batch, 8)
        ko, vo = (torch.empty(290, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in range(2))
        side.wait_stream(torch.cuda.current_stream())
        kept = {t.data_ptr() for t in ins + [into, ws, ko, vo, batch.ctx_len, batch.block_table, batch.q_start]}
        sizes = [t.nbytes for t in ins + [into, ws, ko, vo]]
        P.kv_append(w.c, batch, ins[1], ins[2], q=ins[0], q_out=into, rot=ins[3], g_q=ins[4], g_k=ins[5], stream=side)
        out = P.kv_attention(into, w.c, batch, workspace=ws, stream=side)
        P.kv_read(w.c, batch, k_out=ko, v_out=vo, stream=side)
        return out, kept, sizes
    out, kept, sizes = calls()
    assert not side.query()
    junk = [torch.full((n,), 0xff, dtype=torch.uint8, device="cuda") for n in sizes + [8, 12, 88] for _ in range(2)]
    assert not kept & {t.data_ptr() for t in junk}
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    assert all(torch.equal(a, r) for a, r in zip(P.kv_read(w.c, b), (kr, vr)))
