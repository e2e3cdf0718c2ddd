"""The decode harness over the paged 8-bit cache, against the same block with
the dense bf16 cache and against the decode oracle.

The tolerance is derived for the whole step: an 8-bit cache rounds a key or
value by at most half a step of its page's scale -- int8: 2^-8 of the page's
largest value, about 1/4 of a typical one / 32 = 0.8 % of it in the mean square;
e4m3: 2^-4 of each value at most, 2.6 % in the mean square (uniform between
steps of 2^-3, relative) -- against which the bf16 roundings of the block
(2e-2 bound of the dense harness's test) are kept.  Attention averages keys'
errors out and passes values' errors on at most as they are, and the residual
stream holds more than the attention's output, so twice the values' relative
error is added: 2e-2 + 2 x 0.8e-2 (int8), 2e-2 + 2 x 2.6e-2 (e4m3)."""

import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

SHAPE = dict(n_layers=2, d=256, F=640, n_heads=4, n_kv=2)
BOUND = {"int8": 3.6e-2, "fp8": 7.2e-2}


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _build(ffn, cache, n_seq=1, norm=False, k_in=None, k_ff=None, max_ctx=100):
    from free_ffn_activation_prox_amd.decode import DecodeHarness, DecoderShape, random_layers
    from prox_workloads import gen_weights
    sh = DecoderShape(**SHAPE)
    layers = random_layers(sh, lambda l: gen_weights(77, l, sh.d, sh.F, std=0.05), seed=3, std=0.05)
    if norm:
        g = torch.Generator().manual_seed(9)
        for L in layers:
            L["g_q"], L["g_k"] = ((1 + 0.1 * torch.randn(sh.hd, generator=g)).to(torch.bfloat16).cuda() for _ in range(2))
    return sh, layers, DecodeHarness(sh, layers, max_ctx=max_ctx, ffn=ffn, proxy="int8", k_in=k_in, k_ff=k_ff,
                                     cache=cache, n_seq=n_seq)


def _x(n, d, seed=0):
    return torch.from_numpy(np.random.default_rng(seed).standard_normal((n, d)).astype(np.float32)).cuda()


def _rel(a, b):
    return (torch.linalg.norm(a - b) / torch.linalg.norm(b)).item()


@pytest.mark.parametrize("cache", ["int8", "fp8"])
def test_steps_match_the_oracle(cache):
    from oracle import decode_oracle as D
    from test_gpu_decode import _bf16, _oracle_layers
    sh, layers, h = _build("dense", cache)
    o = D.DecoderOracle(_oracle_layers(layers), sh.n_heads, sh.n_kv, ffn="dense")
    x = _x(1, sh.d)
    for step in range(6):
        xin = x.cpu().numpy()[0].astype(np.float64)
        y = h.step(x)
        ref = o.step(xin, step, rnd=_bf16)
        err = np.linalg.norm(y.cpu().numpy()[0] - ref) / np.linalg.norm(ref)
        print(f"[decode kv] {cache} step {step}: rel L2 error {err:.2e}", flush=True)
        assert err <= BOUND[cache], (step, err)
        x = y


@pytest.mark.parametrize("cache,norm", [("int8", False), ("fp8", True)])
def test_prompt_and_steps_of_several_sequences(cache, norm):
    """A prompt in one pass agrees with the same tokens one by one, and three
    sequences at once with each alone."""
    n = (70, 64, 1)
    xs = [_x(k + 3, SHAPE["d"], seed=k) for k in n]
    sh, _, h = _build("dense", cache, n_seq=3, norm=norm)
    last = [h.prefill(x[:k], seq=s)[-1] for s, (x, k) in enumerate(zip(xs, n))]
    assert h.ctx.tolist() == list(n)
    together = [h.step(torch.stack([x[k + i] for x, k in zip(xs, n)])) for i in range(3)]
    for s, (x, k) in enumerate(zip(xs, n)):
        _, _, one = _build("dense", cache, norm=norm)
        for i in range(k + 3):
            y = one.step(x[i:i + 1])[0]
            if i == k - 1:
                assert _rel(last[s], y) <= BOUND[cache], ("prompt", s)
            if i >= k:
                assert _rel(together[i - k][s], y) <= BOUND[cache], (s, i)


def test_prox_ffn_over_the_paged_cache_and_graph():
    from prox_workloads import pct_count
    d, F = SHAPE["d"], SHAPE["F"]
    k_in, k_ff = pct_count(d, 60), pct_count(F, 30)
    _, _, a = _build("prox", "int8", n_seq=5, k_in=k_in, k_ff=k_ff)
    _, _, b = _build("prox", "int8", n_seq=5, k_in=k_in, k_ff=k_ff)
    xs = [_x(5, d, seed=20 + i) for i in range(8)]
    for h in (a, b):
        h.fill_cache(30, seed=2)
    ref = [a.step(x).clone() for x in xs]
    xin = xs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b.step(xin)
    torch.cuda.current_stream().wait_stream(side)
    b.fill_cache(30, seed=2)
    b.ctx.fill_(30)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        y = b.step(xin)
    for i, x in enumerate(xs):                 # every replay goes on by a token
        xin.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        torch.randn(100, device="cuda").sum().item()
        assert torch.equal(y, ref[i]), i
    assert b.ctx.tolist() == [38] * 5


def test_harness_refusals():
    with pytest.raises(ValueError):
        _build("dense", "dense", n_seq=2)
    with pytest.raises(ValueError):
        _build("dense", "dense", norm=True)
    _, _, h = _build("dense", "dense")
    with pytest.raises(ValueError):
        h.prefill(_x(3, SHAPE["d"]))
    _, _, h = _build("dense", "fp8", max_ctx=10)
    h.prefill(_x(9, SHAPE["d"]))
    h.step(_x(1, SHAPE["d"]))
    with pytest.raises(ValueError):
        h.step(_x(1, SHAPE["d"]))
    with pytest.raises(ValueError):
        h.prefill(_x(1, SHAPE["d"]))
