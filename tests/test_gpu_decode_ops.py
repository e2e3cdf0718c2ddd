"""The decode harness over selected pages, a pool of pages and a shared prefix.

Where every page is kept, or a prefix is shared, the attention's results are the
plain ones up to the rounding of its weights and its bf16 result (2^-8 of a value
at most), which the next layers carry on as they do the block's other bf16
roundings: the 2e-2 bound of the dense harness's test."""

import pytest
import torch

from test_gpu_decode_kv import SHAPE, _rel, _x

pytestmark = pytest.mark.gpu
BOUND = 2e-2


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _build(cache="int8", n_seq=1, max_ctx=600, ffn="dense", **kw):
    from free_ffn_activation_prox_amd.decode import DecodeHarness, DecoderShape, random_layers
    from prox_workloads import gen_weights
    sh = DecoderShape(**SHAPE)
    layers = random_layers(sh, lambda l: gen_weights(77, l, sh.d, sh.F, std=0.05), seed=3, std=0.05)
    return DecodeHarness(sh, layers, max_ctx=max_ctx, ffn=ffn, cache=cache, n_seq=n_seq, **kw)


@pytest.mark.parametrize("cache", ["int8", "fp8"])
def test_every_page_kept_is_the_plain_step(cache):
    plain, picks = _build(cache, n_seq=2), _build(cache, n_seq=2, keep_pages=10)
    for h in (plain, picks):
        h.prefill(_x(300, SHAPE["d"], 1), 0)
        h.prefill(_x(70, SHAPE["d"], 2), 1)
    x = _x(2, SHAPE["d"], 3)
    for _ in range(5):
        a, b = plain.step(x), picks.step(x)
        assert _rel(b, a) <= BOUND
        x = a


def test_few_pages_kept_read_the_pages_that_matter():
    """Keys far larger in one page: the step that keeps 3 pages of 9 sees it."""
    picks = _build(keep_pages=3)
    picks.fill_cache(520)
    for kv in picks.kv:
        kv.k_scale[3] *= 40
    b = picks.step(_x(1, SHAPE["d"], 5))
    assert (picks.picked == 3).any(-1).all() and torch.isfinite(b).all()
    listed = picks.picked[0, 0].tolist()
    assert listed[0] == 0 and listed[-1] == 8 and listed == sorted(listed)


@pytest.mark.parametrize("ffn", ["dense", "prox"])
def test_shared_prefix_is_the_same_prompt_in_every_sequence(ffn):
    d = SHAPE["d"]
    prompt, own = _x(64 * 3 + 5, d, 7), [_x(n, d, 20 + n) for n in (3, 40, 1)]
    kw = dict(ffn=ffn, **({"k_in": d, "k_ff": SHAPE["F"]} if ffn == "prox" else {}))
    a, b = _build(n_seq=3, n_pages=24, **kw), _build(n_seq=3, n_pages=9, **kw)
    ya = [a.prefill(prompt if s == 0 else prompt[:192], s)[-1] for s in range(3)][0]
    yb = b.share_prefix(prompt)[-1]
    assert _rel(yb, ya) <= BOUND and b.ctx.tolist() == [197, 192, 192]
    assert (b.table[:, :3] == b.table[0, :3]).all() and (b.pool.refs[b.table[0, :3].long()] == 3).all()
    for s, x in enumerate(own):
        assert _rel(b.prefill(x, s), a.prefill(x, s)) <= BOUND
    x = _x(3, d, 9)
    for _ in range(4):
        y = a.step(x)
        assert _rel(b.step(x), y) <= BOUND
        x = y
    assert b.status.tolist() == [0, 9 - int((b.pool.refs > 0).sum())]
    assert a.ctx.tolist() == b.ctx.tolist()


@pytest.mark.parametrize("kw", [dict(keep_pages=4), dict(n_pages=30), dict(n_pages=30, share=True), dict(n_pages=30, keep_pages=3)])
def test_captured_step_is_the_eager_step(kw):
    d = SHAPE["d"]
    kw = dict(kw)
    share = kw.pop("share", False)
    hs = [_build(n_seq=2, **kw) for _ in range(2)]
    for h in hs:
        if share:
            h.share_prefix(_x(330, d, 11))
        else:
            h.prefill(_x(330, d, 11), 0)
            h.prefill(_x(90, d, 12), 1)
    eager, h = hs
    xs = [_x(2, d, 30 + i) for i in range(8)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        y = h.step(xs[0])
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(y, eager.step(xs[0]))
    buf = xs[1].clone()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = h.step(buf)
    for x in xs[1:]:
        buf.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, eager.step(x))
    assert h.ctx.tolist() == eager.ctx.tolist()


def test_refusals():
    with pytest.raises(ValueError):
        _build("dense", keep_pages=4)
    with pytest.raises(ValueError):
        _build("dense", n_pages=4)
    with pytest.raises(ValueError):
        _build(keep_pages=1)
    h = _build(n_seq=2, n_pages=5)
    with pytest.raises(ValueError):
        h.prefill(_x(321, SHAPE["d"]), 0)                 # 6 pages
    assert h.ctx.tolist() == [0, 0] and h.lengths == [0, 0]
    h.share_prefix(_x(130, SHAPE["d"]))
    with pytest.raises(ValueError):
        h.share_prefix(_x(10, SHAPE["d"]))
    with pytest.raises(ValueError):
        _build().share_prefix(_x(10, SHAPE["d"]))
