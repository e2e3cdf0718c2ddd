"""Attention over the paged 8-bit cache at the ends of its range: pages that the
table does not name, long runs of pages."""

import numpy as np
import pytest
import torch

from test_gpu_kv import World, f64, settle

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def spare_page_0(w):
    """Take page 0 out of a world's table (before anything is stored)."""
    used = set(int(p) for p in w.table.ravel() if p >= 0)
    free = next(p for p in range(1, w.o.n_pages) if p not in used)
    w.table[w.table == 0] = free


def both(w):
    """The oracle's scales to the GPU's cache."""
    w.c.k_scale.copy_(torch.from_numpy(w.o.ks))
    w.c.v_scale.copy_(torch.from_numpy(w.o.vs))


# ---- pages that the table does not name ------------------------------------------

@pytest.mark.parametrize("kind,H,KV,hd", [("int8", 8, 2, 64), ("fp8", 4, 1, 128)])
def test_pages_that_are_not_there_take_nothing_from_page_0(kind, H, KV, hd):
    w = World(kind, H, KV, hd, [3000, 700, 64], seed=hd)
    spare_page_0(w)
    settle(w, [3000, 700, 64])
    w.table[0, [0, 7, 8, 30]] = -1            # holes: the first page, inside, two in a row
    w.table[1, 3] = w.o.n_pages + 7
    w.table[2, 0] = -5                        # nothing is seen at all
    for new in ([1, 1, 1], [3, 2, 4], [150, 200, 64]):
        b, start = w.batch(new, advance=False)
        q = w.rows(b.n_tokens, H, 1.5)
        w.o.ks[0] = w.o.vs[0] = 0
        both(w)
        want, _ = w.attend(b, start, q=q)
        for scale in (float("inf"), float("nan"), 1e30, 1e-42, -1.0, 5.0):
            w.c.k_scale[0], w.c.v_scale[0] = scale, scale
            assert torch.equal(w.P.kv_attention(q, w.c, b), want), f"page 0 with scale {scale}"


# ---- long runs of pages ------------------------------------------------------------

@pytest.mark.parametrize("kind", ["int8", "fp8"])
def test_sums_stay_exact_over_long_runs_of_pages(kind):
    # 8192 pages and 17 tiles of 256 rows: a block walks some 500 pages on end.
    # All weights are equal (q = 0) and the values whole numbers, +a and -a in
    # turn, so every sum of codes stays below 2^24 and is exact in fp32: the mean
    # over p + 1 positions is rounded by a division, a product and to bf16, at
    # most 2^-8 + 2^-22 of it.
    import free_ffn_activation_prox_amd as P
    n_pages, hd, T = 8192, 64, 17 * 256
    n, top = 64 * n_pages, 127 if kind == "int8" else 448
    rng = np.random.default_rng(53)
    a = rng.integers(1, 16, (n // 2, hd))
    v = np.stack([a, -a], 1).reshape(n_pages, 64, hd)
    v[:, 0], v[:, 1] = top, -top              # every page: scale 1
    v[::64, 3] = 0                            # and 128 of them leave something over
    cache = P.KVCache.alloc(kind, n_pages, 1, hd)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda")[None].contiguous()
    ctx = torch.tensor([n], dtype=torch.int32, device="cuda")
    fill = P.KVBatch(ctx, table, torch.tensor([0, n], dtype=torch.int32, device="cuda"), n_tokens=n)
    vt = torch.from_numpy(v.reshape(n, 1, hd)).to("cuda", torch.bfloat16)
    P.kv_append(cache, fill, vt, vt)
    assert bool((cache.v_scale == 1).all())
    total = np.cumsum(v.reshape(n, hd), 0)[n - T:]
    want = total / np.arange(n - T + 1, n + 1)[:, None]
    for rows in (T, 1):
        b = P.KVBatch(ctx, table, torch.tensor([0, rows], dtype=torch.int32, device="cuda"), n_tokens=rows)
        got = f64(P.kv_attention(torch.zeros(rows, 1, hd, dtype=torch.bfloat16, device="cuda"), cache, b))[:, 0]
        err = np.abs(got - want[T - rows:])
        assert np.all(err <= (2.0 ** -8 + 2.0 ** -22) * np.abs(want[T - rows:])), (rows, float(err.max()))
