"""Attention over the paged 8-bit cache at the ends of its range: pages that the
table does not name."""

import pytest
import torch

from test_gpu_kv import World, settle

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
