"""What the decode harness over the paged 8-bit cache refuses leaves it as it was."""

import pytest
import torch

from test_gpu_decode_kv import SHAPE, _build, _x

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def _state(h):
    return h.lengths[:], h.pos, h.ctx.tolist(), [kv.k.clone() for kv in h.kv]


def _same(a, b):
    return a[:3] == b[:3] and all(torch.equal(x, y) for x, y in zip(a[3], b[3]))


def test_refusals_change_nothing():
    d = SHAPE["d"]
    _, _, h = _build("dense", "int8", n_seq=2, max_ctx=70)
    _, _, twin = _build("dense", "int8", n_seq=2, max_ctx=70)
    for g in (h, twin):
        g.prefill(_x(5, d), seq=1)
        g.step(_x(2, d, seed=1))
    before = _state(h)
    for call in (lambda: h.prefill(_x(3, d), seq=-1), lambda: h.prefill(_x(3, d), seq=2),
                 lambda: h.prefill(_x(3, d + 8)), lambda: h.prefill(_x(70, d)), lambda: h.step(_x(1, d)),
                 lambda: h.step(_x(3, d)), lambda: h.step(_x(2, d - 8)), lambda: h.fill_cache(71)):
        with pytest.raises(ValueError):
            call()
        assert _same(_state(h), before)
    x = _x(2, d, seed=2)
    assert torch.equal(h.step(x), twin.step(x))
