"""The paged 8-bit cache without a GPU: refusals of the C ABI (before anything
is enqueued), the Python handles' checks, and pins of its oracle."""

import ctypes

import numpy as np
import pytest
import torch

import free_ffn_activation_prox_amd as P
from free_ffn_activation_prox_amd import _KVBatch, _KVCache, _KVRotation, _lib
from oracle import kv_oracle as KO

INVALID, UNSUPPORTED, MISMATCH, WORKSPACE = -1, -2, -3, -4
FAKE = 0x10000000      # never dereferenced: every call below fails its checks first


def cache(**over):
    c = _KVCache(1, 10, 2, 128, 128, FAKE, FAKE, FAKE, FAKE)
    for k, v in over.items():
        setattr(c, k, v)
    return c


def batch(**over):
    b = _KVBatch(3, 5, 4, 7, FAKE, FAKE, FAKE)
    for k, v in over.items():
        setattr(b, k, v)
    return b


def rotation(**over):
    r = _KVRotation(FAKE, 7 * 64, 128, 0, None, None, 1e-5)
    for k, v in over.items():
        setattr(r, k, v)
    return r


def append(c=None, b=None, r=None, k=FAKE, ks=256, v=FAKE, vs=256, H=4, q=FAKE, qs=512, qo=FAKE, qos=512):
    return _lib.prox_kv_append(ctypes.byref(c or cache()), ctypes.byref(b or batch()), k, ks, v, vs,
                               ctypes.byref(r or rotation()), H, q, qs, qo, qos, None)


def attend(c=None, b=None, q=FAKE, qs=512, H=4, scale=0.1, window=0, out=2 * FAKE, os=512, ws=FAKE, n=1 << 40):
    return _lib.prox_kv_attention(ctypes.byref(c or cache()), ctypes.byref(b or batch()), q, qs, H, scale, window, out,
                                  os, ws, n, None)


def read(c=None, b=None, k=FAKE, v=FAKE):
    return _lib.prox_kv_read(ctypes.byref(c or cache()), ctypes.byref(b or batch()), k, v, 0, None)


@pytest.mark.parametrize("call", [append, attend, read])
def test_cache_and_batch_refusals(call):
    for over, want in ((dict(kind=0), INVALID), (dict(kind=3), INVALID), (dict(n_pages=0), INVALID),
                       (dict(n_kv=0), INVALID), (dict(n_kv=1025), UNSUPPORTED), (dict(head_dim=0), INVALID),
                       (dict(head_dim=132), INVALID), (dict(head_dim=264), UNSUPPORTED), (dict(head_pad=64), MISMATCH),
                       (dict(k=0), INVALID), (dict(v=0), INVALID), (dict(k_scale=0), INVALID),
                       (dict(v_scale=0), INVALID), (dict(k=FAKE + 8), INVALID), (dict(v_scale=FAKE + 2), INVALID)):
        assert call(c=cache(**over)) == want, over
    for over, want in ((dict(n_seq=0), INVALID), (dict(n_tokens=-1), INVALID), (dict(max_q=-1), INVALID),
                       (dict(n_tokens=(1 << 28) + 1), UNSUPPORTED), (dict(max_pages=0), INVALID),
                       (dict(max_pages=1 << 26), UNSUPPORTED), (dict(ctx_len=0), INVALID),
                       (dict(block_table=0), INVALID), (dict(ctx_len=FAKE + 1), INVALID),
                       (dict(q_start=0), INVALID)):                    # 5 tokens of 3 sequences need q_start
        assert call(b=batch(**over)) == want, over


def test_append_refusals():
    assert append(k=0) == INVALID and append(v=0) == INVALID
    assert append(ks=255) == INVALID and append(ks=260) == INVALID and append(vs=128) == INVALID
    assert append(k=FAKE + 2) == INVALID
    assert append(q=0) == INVALID and append(qo=0) == INVALID
    assert append(H=3) == INVALID and append(H=0) == INVALID and append(H=2048) == UNSUPPORTED
    assert append(qs=504) == INVALID and append(qos=504) == INVALID
    assert append(qs=520, qos=528) == INVALID                          # in place with two strides
    for over, want in ((dict(rot=FAKE + 4), INVALID), (dict(rot_dim=0), INVALID), (dict(rot_dim=127), INVALID),
                       (dict(rot_dim=130), INVALID), (dict(pairing=2), INVALID),
                       (dict(pairing=1, rot_dim=40), UNSUPPORTED), (dict(rot_rows=447), INVALID),
                       (dict(g_q=FAKE, eps=-1.0), INVALID), (dict(g_k=FAKE, eps=float("nan")), INVALID),
                       (dict(g_k=FAKE + 2), INVALID)):
        assert append(r=rotation(**over)) == want, over
    assert b"table" in (append(r=rotation(rot_rows=447)), _lib.prox_last_error())[1]


def test_attention_refusals():
    assert attend(q=0) == INVALID and attend(out=0) == INVALID and attend(out=FAKE) == INVALID
    assert attend(H=5) == INVALID and attend(H=1026) == UNSUPPORTED
    assert attend(qs=511) == INVALID and attend(os=500) == INVALID
    assert attend(scale=float("inf")) == INVALID and attend(scale=float("nan")) == INVALID
    assert attend(window=-1) == INVALID
    assert attend(ws=0) == INVALID and attend(ws=FAKE + 16) == INVALID
    assert attend(n=0) == WORKSPACE and b"workspace" in _lib.prox_last_error()


def test_read_refusals():
    assert read(k=0) == INVALID and read(v=0) == INVALID and read(k=FAKE + 8) == INVALID


def test_nothing_to_do_is_no_error():
    for b in (batch(n_tokens=0), batch(max_q=0)):
        assert append(b=b) == 0 and attend(b=b) == 0 and read(b=b) == 0


def test_sizes():
    assert [P.kv_head_pad(d) for d in (8, 64, 72, 128, 200, 256)] == [64, 64, 128, 128, 256, 256]
    assert [P.kv_head_pad(d) for d in (0, -8, 4, 100, 264)] == [0] * 5
    assert _lib.prox_kv_workspace_bytes(ctypes.byref(cache()), ctypes.byref(batch()), 4) > 0
    assert _lib.prox_kv_workspace_bytes(ctypes.byref(cache()), ctypes.byref(batch()), 3) == 0
    assert _lib.prox_kv_workspace_bytes(ctypes.byref(cache(kind=9)), ctypes.byref(batch()), 4) == 0


def test_python_handles_refuse_host_tensors():
    z = torch.zeros(2, 2, 64 * 64, dtype=torch.uint8)
    sc = torch.zeros(2, 2)
    with pytest.raises(ValueError):
        P.KVCache("int8", 64, z, z, sc, sc)
    with pytest.raises(ValueError):
        P.KVCache("int4", 64, z, z, sc, sc)
    i = torch.zeros(3, dtype=torch.int32)
    with pytest.raises(ValueError):
        P.KVBatch(i, torch.zeros(3, 4, dtype=torch.int32))
    with pytest.raises(ValueError):
        P.KVBatch(i, torch.zeros(2, 4, dtype=torch.int32))


# ---- pins of the oracle ---------------------------------------------------------

def test_e4m3_table_is_the_type():
    codes = np.arange(256, dtype=np.uint8)
    want = torch.from_numpy(codes).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(KO.decode("fp8", codes), want, equal_nan=True)
    assert np.array_equal(KO.decode("int8", codes), codes.view(np.int8))


def test_encode_against_torch():
    x = np.concatenate([np.random.default_rng(0).standard_normal(4000) * s for s in (1e-3, 0.1, 3.0, 100.0)]
                       + [np.arange(-450, 450) * 0.5, KO._E4M3, (KO._E4M3[1:] + KO._E4M3[:-1]) / 2]).astype(np.float32)
    t = torch.from_numpy(x)
    assert np.array_equal(KO.encode("fp8", x), t.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8).numpy())
    assert np.array_equal(KO.encode("int8", x), t.clamp(-127, 127).round().to(torch.int8).view(torch.uint8).numpy())
    assert list(KO.encode("int8", np.array([0.5, 1.5, -2.5, np.nan, np.inf, -np.inf]))) == [0, 2, 254, 0, 127, 129]


def test_layout_of_a_page_by_hand():
    c = KO.Cache("int8", 1, 1, 128)
    t = np.zeros((1, 1, 64, 128), np.uint8)
    t[0, 0, 37, 77] = 5            # slot 37 = 16 * 2 + 5; channel 77 = 64 + 0 * 16 + 13 = 16 * 4 + 13
    c.put("k", t)
    assert np.flatnonzero(c.k).tolist() == [(((1 * 4 + 2) * 4 + 0) * 16 + 5) * 16 + 13]
    assert np.array_equal(c.tokens("k"), t)
    c.put("v", t)                  # slot 37 = 16 * 2 + 4 * 1 + 1
    assert np.flatnonzero(c.v).tolist() == [(((4 * 4 + 1) * 16 + 13) * 4 + 2) * 4 + 1]
    assert np.array_equal(c.tokens("v"), t)


def test_rotation_turns_and_keeps_length():
    rng = np.random.default_rng(1)
    x = rng.standard_normal((3, 16))
    ang = np.arange(5)[:, None] * 0.3 ** np.arange(4)[None]
    rot = np.stack([np.cos(ang), np.sin(ang)], -1).astype(np.float32)
    for pairing in ("interleaved", "halves"):
        y = KO.turn(x, 3, rot, pairing, None, 0.0)
        assert np.array_equal(y[:, 8:], x[:, 8:])                       # channels past rot_dim pass
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1), rtol=1e-6)
        assert np.array_equal(KO.turn(x, 0, rot, pairing, None, 0.0), x)
    z = KO.turn(x, 2, rot, "halves", None, 0.0)
    assert np.allclose(z[:, 1], x[:, 1] * np.cos(0.6) - x[:, 5] * np.sin(0.6), atol=1e-6)


def test_append_grows_scale_once_and_is_idempotent():
    rng = np.random.default_rng(2)
    for kind in ("int8", "fp8"):
        c = KO.Cache(kind, 3, 1, 16)
        table = np.array([[2]], np.int32)
        k = rng.standard_normal((3, 1, 16)).astype(np.float32).astype(np.float64)
        k[2] *= 4
        KO.append(c, table, [2], [0, 2], 9, k[:2], k[:2])
        s0 = c.ks[2, 0]
        KO.append(c, table, [3], [0, 1], 9, k[2:], k[2:])
        assert c.ks[2, 0] > s0 and not c.k[:2].any()
        back = KO.gather(c, table, 0, 0, 3)[0]
        step = c.ks[2, 0] * (1.0 if kind == "int8" else 32.0)           # the largest step of a code
        assert np.max(np.abs(back - k)) <= 1.5 * step                    # rounded at most twice
        before = c.k.copy(), c.ks.copy()
        KO.append(c, table, [3], [0, 1], 9, k[2:], k[2:])
        assert np.array_equal(c.k, before[0]) and np.array_equal(c.ks, before[1])


def test_attention_of_one_visible_key_is_its_value():
    rng = np.random.default_rng(3)
    c = KO.Cache("int8", 2, 1, 8)
    table = np.array([[1, 0]], np.int32)
    k = rng.standard_normal((70, 1, 8))
    KO.append(c, table, [70], [0, 70], 70, k, k)
    o, _ = KO.attention(c, table, [70], [0, 70], 70, rng.standard_normal((70, 2, 8)), 0.3, window=1)
    v = KO.gather(c, table, 0, 0, 70)[1]
    assert np.allclose(o, np.repeat(v, 2, axis=1))
    full, _ = KO.attention(c, table, [70], [0, 70], 70, np.zeros((70, 2, 8)), 0.3)
    assert np.allclose(full[:, 0], np.cumsum(v[:, 0], 0) / np.arange(1, 71)[:, None])
