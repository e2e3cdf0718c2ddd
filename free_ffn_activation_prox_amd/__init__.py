"""Prox sparse SwiGLU FFN decode path on MI355X — thin Python binding.

Argument marshalling over the C ABI in ``include/prox.h`` (ctypes).  Every
step of the path runs in the HIP library ``libprox_hip.so``; torch only
provides device memory and the stream.  Importing fails loudly when the
library has not been built (``python -m free_ffn_activation_prox_amd.build``).

Method: "Prox: Training-Free FFN Activation Sparsity via Approximate
Intermediate-Channel Salience in LLMs", Abstract (two stages: input-sparse
quantized proxy -> shared channel mask -> exact sparse SwiGLU).
"""

from __future__ import annotations

import contextlib
import ctypes
import os
from dataclasses import dataclass
from typing import Dict, Optional, Tuple

# torch first: the library then binds to the HIP runtime torch has loaded, so
# the process holds one runtime (one device context) whichever module a
# program imports first.
import torch  # noqa: F401

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libprox_hip.so")

PROX_OK = 0
KINDS = {"int8": 1, "int4": 2, "exact": 3}


class ProxError(RuntimeError):
    def __init__(self, status: int, where: str, detail: str):
        self.status = status
        super().__init__(f"{where}: {_status_str(status)}: {detail}")


class _Weights(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("w_gate_t", ctypes.c_void_p), ("w_up_t", ctypes.c_void_p),
                ("w_down", ctypes.c_void_p)]


class _Proxy(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32),
                ("f_pad", ctypes.c_int32), ("groups", ctypes.c_int32), ("tile_ch", ctypes.c_int32),
                ("row_stride", ctypes.c_size_t), ("scale_offset", ctypes.c_size_t),
                ("bytes", ctypes.c_size_t), ("buf", ctypes.c_void_p)]


class _QWeights(ctypes.Structure):
    _fields_ = [("d_model", ctypes.c_int32), ("d_ff", ctypes.c_int32), ("scale_offset", ctypes.c_size_t),
                ("bytes", ctypes.c_size_t), ("buf", ctypes.c_void_p)]


class _Taps(ctypes.Structure):
    _fields_ = [("in_idx", ctypes.c_void_p), ("key", ctypes.c_void_p), ("h_hat", ctypes.c_void_p),
                ("events", ctypes.POINTER(ctypes.c_void_p)), ("n_events", ctypes.c_int32),
                ("event_mode", ctypes.c_int32), ("stream_idx", ctypes.c_void_p), ("timeline", ctypes.c_void_p)]


class _KVCache(ctypes.Structure):
    _fields_ = [("kind", ctypes.c_int32), ("n_pages", ctypes.c_int32), ("n_kv", ctypes.c_int32),
                ("head_dim", ctypes.c_int32), ("head_pad", ctypes.c_int32), ("k", ctypes.c_void_p),
                ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p), ("v_scale", ctypes.c_void_p)]


class _KVBatch(ctypes.Structure):
    _fields_ = [("n_seq", ctypes.c_int32), ("n_tokens", ctypes.c_int32), ("max_q", ctypes.c_int32),
                ("max_pages", ctypes.c_int32), ("ctx_len", ctypes.c_void_p), ("block_table", ctypes.c_void_p),
                ("q_start", ctypes.c_void_p)]


class _KVRotation(ctypes.Structure):
    _fields_ = [("rot", ctypes.c_void_p), ("rot_rows", ctypes.c_int32), ("rot_dim", ctypes.c_int32),
                ("pairing", ctypes.c_int32), ("g_q", ctypes.c_void_p), ("g_k", ctypes.c_void_p),
                ("eps", ctypes.c_float)]


N_PHASES = 3
PHASES = ("stage1", "stage2", "reduce_y")


def _load() -> ctypes.CDLL:
    if not os.path.exists(LIB_PATH):
        raise ImportError(f"Prox HIP library missing: {LIB_PATH}; build it with "
                          "`python -m free_ffn_activation_prox_amd.build`")
    lib = ctypes.CDLL(LIB_PATH)
    P, I32, I64, SZ = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64, ctypes.c_size_t
    sig = {
        "prox_abi_version": (I32, []),
        "prox_proxy_bytes": (SZ, [I32, I32, I32]),
        "prox_build_proxy": (I32, [ctypes.POINTER(_Weights), I32, P, SZ, ctypes.POINTER(_Proxy), P]),
        "prox_workspace_bytes": (SZ, [I32, I32, I32, I32]),
        "prox_ffn_forward": (I32, [P, I32, ctypes.POINTER(_Weights), ctypes.POINTER(_Proxy), I32, I32,
                                   P, P, P, P, SZ, P]),
        "prox_ffn_forward_taps": (I32, [P, I32, ctypes.POINTER(_Weights), ctypes.POINTER(_Proxy), I32,
                                        I32, P, P, P, P, SZ, ctypes.POINTER(_Taps), P]),
        "prox_noalloc_scratch_bytes": (SZ, []),
        "prox_ffn_forward_noalloc": (I32, [P, I32, ctypes.POINTER(_Weights), ctypes.POINTER(_Proxy), I32, I32,
                                           P, P, P, P]),
        "prox_read_probe": (I32, [P, SZ, P, I32, P]),
        "prox_quality": (I32, [P, P, I32, I32, P, P, I32, P, P, P]),
        "prox_qweights_bytes": (SZ, [I32, I32]),
        "prox_build_qweights": (I32, [ctypes.POINTER(_Weights), P, SZ, ctypes.POINTER(_QWeights), P]),
        "prox_ffn_forward_q8": (I32, [P, I32, ctypes.POINTER(_QWeights), ctypes.POINTER(_Proxy), I32, I32, P, P, P,
                                      P, SZ, ctypes.POINTER(_Taps), P]),
        "prox_kv_head_pad": (I32, [I32]),
        "prox_kv_append": (I32, [ctypes.POINTER(_KVCache), ctypes.POINTER(_KVBatch), P, I64, P, I64,
                                 ctypes.POINTER(_KVRotation), I32, P, I64, P, I64, P]),
        "prox_kv_workspace_bytes": (SZ, [ctypes.POINTER(_KVCache), ctypes.POINTER(_KVBatch), I32]),
        "prox_kv_attention": (I32, [ctypes.POINTER(_KVCache), ctypes.POINTER(_KVBatch), P, I64, I32, ctypes.c_float,
                                    I32, P, I64, P, SZ, P]),
        "prox_kv_read": (I32, [ctypes.POINTER(_KVCache), ctypes.POINTER(_KVBatch), P, P, I32, P]),
        "prox_status_str": (ctypes.c_char_p, [I32]),
        "prox_last_error": (ctypes.c_char_p, []),
    }
    for name, (res, args) in sig.items():
        fn = getattr(lib, name)
        fn.restype, fn.argtypes = res, args
    return lib


_lib = _load()


def _status_str(st: int) -> str:
    return _lib.prox_status_str(st).decode()


def _check(st: int, where: str) -> None:
    if st != PROX_OK:
        raise ProxError(st, where, _lib.prox_last_error().decode())


def abi_version() -> int:
    return _lib.prox_abi_version()


def library_sha256() -> str:
    """sha256 (first 16 hex digits) of the loaded library file."""
    import hashlib
    with open(LIB_PATH, "rb") as fh:
        return hashlib.sha256(fh.read()).hexdigest()[:16]


def proxy_bytes(d_model: int, d_ff: int, kind: str) -> int:
    return _lib.prox_proxy_bytes(d_model, d_ff, KINDS[kind])


def workspace_bytes(d_model: int, d_ff: int, batch: int, kind: str) -> int:
    return _lib.prox_workspace_bytes(d_model, d_ff, batch, KINDS[kind])


def _stream_ptr(stream) -> Optional[int]:
    import torch
    s = stream if stream is not None else torch.cuda.current_stream()
    return s.cuda_stream


@dataclass
class Weights:
    """bf16 device tensors: w_gate_t, w_up_t [d_ff][d_model]; w_down [d_ff][d_model]."""

    w_gate_t: "object"
    w_up_t: "object"
    w_down: "object"

    def __post_init__(self):
        import torch
        for n in ("w_gate_t", "w_up_t", "w_down"):
            t = getattr(self, n)
            if t.dtype != torch.bfloat16 or not t.is_cuda or not t.is_contiguous() or t.dim() != 2:
                raise ValueError(f"{n} must be a contiguous 2-D bf16 CUDA tensor")
        F, d = self.w_gate_t.shape
        if tuple(self.w_up_t.shape) != (F, d) or tuple(self.w_down.shape) != (F, d):
            raise ValueError("w_gate_t, w_up_t and w_down must all be [d_ff][d_model]")
        self.d_ff, self.d_model = int(F), int(d)
        self._c = _Weights(self.d_model, self.d_ff, self.w_gate_t.data_ptr(),
                           self.w_up_t.data_ptr(), self.w_down.data_ptr())


@dataclass
class Proxy:
    kind: str
    buf: "object"          # uint8 device tensor owning the proxy bytes
    desc: _Proxy

    @property
    def f_pad(self) -> int:
        return self.desc.f_pad

    def codes_and_scales(self):
        """Device views: codes [tiles][d][128] uint8, scales [2][groups][f_pad] fp32."""
        import torch
        d, fp, tc = self.desc.d_model, self.desc.f_pad, self.desc.tile_ch
        codes = self.buf[: (fp // tc) * d * 128].view(fp // tc, d, 128)
        n = 2 * self.desc.groups * fp
        so = self.desc.scale_offset
        scales = self.buf[so: so + 4 * n].view(torch.float32).view(2, self.desc.groups, fp)
        return codes, scales


def build_proxy(weights: Weights, kind: str, stream=None) -> Proxy:
    """Quantized proxy of W_gate / W_up (one-time, training-free).  kind
    "exact" (exact-mask mode) builds nothing: the weights rank themselves."""
    import torch
    if kind == "exact":
        desc = _Proxy()
        _check(_lib.prox_build_proxy(ctypes.byref(weights._c), KINDS[kind], None, 0, ctypes.byref(desc),
                                     _stream_ptr(stream)), "prox_build_proxy")
        return Proxy(kind, None, desc)
    nbytes = proxy_bytes(weights.d_model, weights.d_ff, kind)
    if nbytes == 0:
        raise ValueError("invalid shape/kind for a proxy")
    buf = torch.empty(nbytes + 256, dtype=torch.uint8, device=weights.w_gate_t.device)
    off = (-buf.data_ptr()) % 256
    buf = buf[off: off + nbytes]
    desc = _Proxy()
    _check(_lib.prox_build_proxy(ctypes.byref(weights._c), KINDS[kind], buf.data_ptr(), nbytes,
                                 ctypes.byref(desc), _stream_ptr(stream)), "prox_build_proxy")
    return Proxy(kind, buf, desc)


@dataclass
class QWeights:
    """Quantized Stage-2 weights: int8 rows of W_gate^T, W_up^T, W_down and
    their fp32 scales in one device buffer (prox_build_qweights)."""

    buf: "object"
    desc: _QWeights

    @property
    def d_model(self) -> int:
        return self.desc.d_model

    @property
    def d_ff(self) -> int:
        return self.desc.d_ff

    def codes_and_scales(self):
        """Device views: codes [3][F][d] int8, scales [3][F] fp32."""
        import torch
        d, F = self.desc.d_model, self.desc.d_ff
        codes = self.buf[: 3 * F * d].view(torch.int8).view(3, F, d)
        so = self.desc.scale_offset
        scales = self.buf[so: so + 12 * F].view(torch.float32).view(3, F)
        return codes, scales


def qweights_bytes(d_model: int, d_ff: int) -> int:
    return _lib.prox_qweights_bytes(d_model, d_ff)


def build_qweights(weights: Weights, stream=None) -> QWeights:
    import torch
    n = qweights_bytes(weights.d_model, weights.d_ff)
    if n == 0:
        raise ValueError("invalid shape for quantized weights")
    raw = torch.empty(n + 256, dtype=torch.uint8, device=weights.w_gate_t.device)
    off = (-raw.data_ptr()) % 256
    buf = raw[off: off + n]
    desc = _QWeights()
    _check(_lib.prox_build_qweights(ctypes.byref(weights._c), buf.data_ptr(), n, ctypes.byref(desc),
                                    _stream_ptr(stream)), "prox_build_qweights")
    return QWeights(buf, desc)


def alloc_workspace(d_model: int, d_ff: int, batch: int, kind: str, device="cuda"):
    import torch
    n = workspace_bytes(d_model, d_ff, batch, kind)
    if n == 0:
        raise ValueError("invalid shape/batch for a workspace")
    # scratch: its contents on entry do not matter
    raw = torch.empty(n + 256, dtype=torch.uint8, device=device)
    off = (-raw.data_ptr()) % 256
    return raw[off: off + n]


def ffn_forward(x, weights, proxy: Proxy, k_in: int, k_ff: int, *, y=None, mask=None,
                idx=None, workspace=None, taps: bool = False, events=None, kernel_events: bool = False,
                stream=None):
    """Sparse SwiGLU forward for x [B][d] bf16.  Returns (y fp32 [B][d], mask u8 [B][F],
    idx int32 [B][k_ff]) and, with ``taps``, a dict of in_idx / key / h_hat.
    ``events`` (measurement hook): torch.cuda.Event(enable_timing=True) objects
    already recorded once, or raw hipEvent_t handles (int).  By default
    N_PHASES + 1 events recorded at the phase boundaries on the launch stream;
    with ``kernel_events``, 2 * N_PHASES events carried by the kernels
    themselves: events[2p] .. events[2p + 1] spans phase p's kernels alone."""
    import torch
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous() or x.dim() != 2:
        raise ValueError("x must be a contiguous 2-D bf16 CUDA tensor")
    B, d = x.shape
    F = weights.d_ff
    dev = x.device
    q8 = isinstance(weights, QWeights)
    if y is None:
        y = torch.empty(B, d, dtype=torch.float32, device=dev)
    if mask is None:
        mask = torch.empty(B, F, dtype=torch.uint8, device=dev)
    if idx is None:
        idx = torch.empty(B, max(k_ff, 1), dtype=torch.int32, device=dev)
    if workspace is None:
        workspace = alloc_workspace(d, F, B, proxy.kind, dev)
    sp = _stream_ptr(stream)
    if events is not None:
        arr = (ctypes.c_void_p * len(events))(*[getattr(e, "cuda_event", e) for e in events])
        ct = _Taps(None, None, None, arr, len(events), 1 if kernel_events else 0, None, None)
        _call_forward(q8, x, B, weights, proxy, k_in, k_ff, y, mask, idx, workspace, ct, sp)
        return y, mask, idx[:, :k_ff]
    if taps:
        t = {"in_idx": torch.empty(B, max(k_in, 1), dtype=torch.int32, device=dev),
             "key": torch.empty(B, F, dtype=torch.float32, device=dev),
             "h_hat": torch.empty(B, F, dtype=torch.float64, device=dev),
             "stream_idx": torch.full((B, max(k_ff, 1)), -1, dtype=torch.int32, device=dev)}
        ct = _Taps(t["in_idx"].data_ptr(), t["key"].data_ptr(), t["h_hat"].data_ptr(), None, 0, 0,
                   t["stream_idx"].data_ptr(), None)
        _call_forward(q8, x, B, weights, proxy, k_in, k_ff, y, mask, idx, workspace, ct, sp)
        t["in_idx"] = t["in_idx"][:, :k_in]
        t["stream_idx"] = t["stream_idx"][:, :k_ff]
        return y, mask, idx[:, :k_ff], t
    if q8:
        _call_forward(True, x, B, weights, proxy, k_in, k_ff, y, mask, idx, workspace, None, sp)
    else:
        _check(_lib.prox_ffn_forward(x.data_ptr(), B, ctypes.byref(weights._c), ctypes.byref(proxy.desc),
                                     k_in, k_ff, y.data_ptr(), mask.data_ptr(), idx.data_ptr(),
                                     workspace.data_ptr(), workspace.numel(), sp),
               "prox_ffn_forward")
    return y, mask, idx[:, :k_ff]


def _call_forward(q8, x, B, weights, proxy, k_in, k_ff, y, mask, idx, workspace, ct, sp):
    tp = ctypes.byref(ct) if ct is not None else None
    if q8:
        _check(_lib.prox_ffn_forward_q8(x.data_ptr(), B, ctypes.byref(weights.desc), ctypes.byref(proxy.desc), k_in,
                                        k_ff, y.data_ptr(), mask.data_ptr(), idx.data_ptr(), workspace.data_ptr(),
                                        workspace.numel(), tp, sp),
               "prox_ffn_forward_q8")
    else:
        _check(_lib.prox_ffn_forward_taps(x.data_ptr(), B, ctypes.byref(weights._c), ctypes.byref(proxy.desc),
                                          k_in, k_ff, y.data_ptr(), mask.data_ptr(), idx.data_ptr(),
                                          workspace.data_ptr(), workspace.numel(), tp, sp),
               "prox_ffn_forward_taps")


def read_probe(buf, sink, blocks: int, stream=None) -> None:
    """Measurement helper: one plain streaming read of the device tensor `buf`
    (prox_read_probe); `sink` is an int32/uint32 device tensor of blocks * 512."""
    if sink.numel() < blocks * 512:
        raise ValueError("sink needs blocks * 512 words")
    _check(_lib.prox_read_probe(buf.data_ptr(), buf.numel() * buf.element_size(), sink.data_ptr(), blocks,
                                _stream_ptr(stream)), "prox_read_probe")


def timeline_forward(x, weights: Weights, proxy: Proxy, k_in: int, k_ff: int, *, y, mask, idx, workspace,
                     stream=None):
    """Measurement hook: the forward with the per-block timeline tap; returns
    the uint64 device tensor [2][1024][8] of 100 MHz counter stamps."""
    import torch
    tl = torch.zeros(2 * 1024 * 8, dtype=torch.int64, device=x.device)
    ct = _Taps(None, None, None, None, 0, 0, None, tl.data_ptr())
    B = x.shape[0]
    _check(_lib.prox_ffn_forward_taps(x.data_ptr(), B, ctypes.byref(weights._c), ctypes.byref(proxy.desc), k_in,
                                      k_ff, y.data_ptr(), mask.data_ptr(), idx.data_ptr(), workspace.data_ptr(),
                                      workspace.numel(), ctypes.byref(ct), _stream_ptr(stream)),
           "prox_ffn_forward_taps")
    return tl.view(2, 1024, 8)


def quality(mask_a, mask_b, y, y_ref, stream=None):
    """Quality diagnostics (prox_quality) on device tensors: per token, the kept
    channels two masks share (uint8 [B][F] each) and ||y - y_ref|| / ||y_ref||
    (fp32 [B][d] each).  Returns (overlap int32 [B], err float64 [B])."""
    import torch
    B, F = mask_a.shape
    d = y.shape[1]
    for t, dt in ((mask_a, torch.uint8), (mask_b, torch.uint8), (y, torch.float32), (y_ref, torch.float32)):
        if t.dtype != dt or not t.is_contiguous() or t.shape[0] != B:
            raise ValueError("quality: wrong dtype, layout or batch")
    overlap = torch.empty(B, dtype=torch.int32, device=y.device)
    err = torch.empty(B, dtype=torch.float64, device=y.device)
    _check(_lib.prox_quality(mask_a.data_ptr(), mask_b.data_ptr(), B, F, y.data_ptr(), y_ref.data_ptr(), d,
                             overlap.data_ptr(), err.data_ptr(), _stream_ptr(stream)), "prox_quality")
    return overlap, err


def noalloc_scratch_bytes() -> int:
    return _lib.prox_noalloc_scratch_bytes()


def ffn_forward_noalloc(x, weights: Weights, proxy: Proxy, k_in: int, k_ff: int, *, y, mask, idx,
                        stream=None):
    """prox_ffn_forward_noalloc: the forward with the library's fixed device
    scratch as workspace (no allocation in the call).  y, mask and idx are the
    caller's ([B][d] fp32, [B][F] uint8, [B][>= max(k_ff, 1)] int32)."""
    import torch
    if x.dtype != torch.bfloat16 or not x.is_cuda or not x.is_contiguous() or x.dim() != 2:
        raise ValueError("x must be a contiguous 2-D bf16 CUDA tensor")
    B, d = x.shape
    for t, dt, shape in ((y, torch.float32, (B, d)), (mask, torch.uint8, (B, weights.d_ff))):
        if t.dtype != dt or tuple(t.shape) != shape or not t.is_contiguous():
            raise ValueError("y / mask: wrong dtype, shape or layout")
    if idx.dtype != torch.int32 or idx.dim() != 2 or idx.shape[0] != B or idx.shape[1] < max(k_ff, 1) \
            or not idx.is_contiguous():
        raise ValueError("idx must be int32 [B][>= max(k_ff, 1)]")
    _check(_lib.prox_ffn_forward_noalloc(x.data_ptr(), B, ctypes.byref(weights._c), ctypes.byref(proxy.desc),
                                         k_in, k_ff, y.data_ptr(), mask.data_ptr(), idx.data_ptr(),
                                         _stream_ptr(stream)),
           "prox_ffn_forward_noalloc")
    return y, mask, idx[:, :k_ff]


# ---- paged 8-bit key/value cache ------------------------------------------------

KV_KINDS = {"int8": 1, "fp8": 2}
KV_PAGE = 64
ROPE_PAIRINGS = {"interleaved": 0, "halves": 1}


def kv_head_pad(head_dim: int) -> int:
    """Channels a head takes in the cache (head_dim rounded up to a multiple of 64)."""
    return _lib.prox_kv_head_pad(head_dim)


def _need(ok: bool, what: str) -> None:
    if not ok:
        raise ValueError(what)


def _on(stream, device):
    """(stream pointer, whether the device is the current one) of a call on
    tensors of `device`: the given stream (the caller's inputs must be ready on
    it; they may be let go of once the call returns), else the device's current
    one."""
    if stream is None:
        return _raw_stream(device.index), _current_device() == device.index
    if stream.device != device:
        raise ValueError("stream and tensors are on different devices")
    return stream.cuda_stream, _current_device() == device.index


# the current stream's handle and the current device, without the objects that
# torch.cuda makes around them (2 us a call)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _kv_call(fn, where, device, here, *args):
    """One call of the library with `device` as the current device."""
    if here:
        st = fn(*args)
    else:
        with torch.cuda.device(device):
            st = fn(*args)
    if st != PROX_OK:
        _check(st, where)


def _made_on(stream):
    """Context in which a call's own tensors are allocated: the stream that the
    call runs on, so that their memory is that stream's."""
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _held_for(stream, cache, batch, *tensors):
    """After a call on a given stream: the memory of what it reads and writes
    stays until that stream has run it, whatever the caller lets go of."""
    if stream is not None and stream.cuda_stream != _raw_stream(cache.device.index):
        for t in (cache.k, cache.v, cache.k_scale, cache.v_scale, batch.ctx_len, batch.block_table, batch.q_start) + tensors:
            if t is not None:
                t.record_stream(stream)


class KVCache:
    """Handle of a paged 8-bit key/value cache (layout: ``include/prox.h``).

    kind "int8" or "fp8" (e4m3); device tensors k, v uint8 [n_pages][n_kv]
    [64 * kv_head_pad(head_dim)] and k_scale, v_scale fp32 [n_pages][n_kv].
    ``KVCache.alloc`` makes an empty one."""

    def __init__(self, kind: str, head_dim: int, k, v, k_scale, v_scale):
        _need(kind in KV_KINDS, f"unknown cache kind {kind!r}")
        hp = kv_head_pad(head_dim)
        _need(hp > 0, "head_dim must be a multiple of 8 between 8 and 256")
        _need(k.dim() == 3 and k.shape[2] == KV_PAGE * hp, "k must be [n_pages][n_kv][64 * kv_head_pad(head_dim)]")
        for n, t, dt, shape in (("k", k, torch.uint8, k.shape), ("v", v, torch.uint8, k.shape),
                                ("k_scale", k_scale, torch.float32, k.shape[:2]),
                                ("v_scale", v_scale, torch.float32, k.shape[:2])):
            _need(t.dtype == dt and t.is_cuda and t.is_contiguous() and t.shape == shape and t.device == k.device,
                  f"{n}: wrong dtype, shape, layout or device")
        self.kind, self.head_dim, self.head_pad = kind, int(head_dim), hp
        self.n_pages, self.n_kv = int(k.shape[0]), int(k.shape[1])
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.device = k.device
        self._c = _KVCache(KV_KINDS[kind], self.n_pages, self.n_kv, self.head_dim, hp, k.data_ptr(), v.data_ptr(),
                           k_scale.data_ptr(), v_scale.data_ptr())
        self._ref = ctypes.byref(self._c)

    @classmethod
    def alloc(cls, kind: str, n_pages: int, n_kv: int, head_dim: int, device="cuda") -> "KVCache":
        hp = kv_head_pad(head_dim)
        _need(hp > 0, "head_dim must be a multiple of 8 between 8 and 256")
        codes = [torch.zeros(n_pages, n_kv, KV_PAGE * hp, dtype=torch.uint8, device=device) for _ in range(2)]
        scales = [torch.zeros(n_pages, n_kv, dtype=torch.float32, device=device) for _ in range(2)]
        return cls(kind, head_dim, *codes, *scales)


class KVBatch:
    """The tokens a call works on: the last tokens of n_seq sequences.

    ctx_len int32 [n_seq]: tokens of each sequence, the call's included;
    block_table int32 [n_seq][max_pages]: pages of each sequence in order;
    q_start int32 [n_seq + 1]: rows of the call (None: one row per sequence);
    n_tokens: rows; max_q: the most rows of one sequence (default n_tokens).
    The device tensors are read when the kernels run."""

    def __init__(self, ctx_len, block_table, q_start=None, *, n_tokens: Optional[int] = None,
                 max_q: Optional[int] = None):
        n_seq = int(ctx_len.shape[0])
        _need(block_table.dim() == 2 and block_table.shape[0] == n_seq, "block_table must be [n_seq][max_pages]")
        _need(q_start is not None or n_tokens in (None, n_seq), "without q_start there is one token per sequence")
        _need(q_start is None or n_tokens is not None, "n_tokens is needed with q_start")
        for n, t, shape in (("ctx_len", ctx_len, (n_seq,)), ("block_table", block_table, tuple(block_table.shape)),
                            ("q_start", q_start, (n_seq + 1,))):
            if t is not None:
                _need(t.dtype == torch.int32 and t.is_cuda and t.is_contiguous() and tuple(t.shape) == shape
                      and t.device == ctx_len.device, f"{n}: must be int32, contiguous, of shape {shape}, on one device")
        self.n_seq, self.n_tokens = n_seq, n_seq if n_tokens is None else int(n_tokens)
        self.max_q = (1 if q_start is None else self.n_tokens) if max_q is None else int(max_q)
        _need(max(n_seq, self.n_tokens, self.max_q, int(block_table.shape[1])) < 1 << 31, "sizes must be below 2^31")
        self.ctx_len, self.block_table, self.q_start = ctx_len, block_table, q_start
        self.device = ctx_len.device
        self._c = _KVBatch(n_seq, self.n_tokens, self.max_q, int(block_table.shape[1]), ctx_len.data_ptr(),
                           block_table.data_ptr(), 0 if q_start is None else q_start.data_ptr())
        self._ref = ctypes.byref(self._c)


def _kv_rows(name, t, n, heads, hd, device):
    """Row stride of an activation [n][heads][hd] (heads adjacent); of one row it says nothing."""
    shape, stride = t.shape, t.stride()
    if t.dtype is not torch.bfloat16 or t.device != device:
        raise ValueError(f"{name} must be bf16 on the cache's device")
    if len(shape) != 3 or shape[0] != n or shape[2] != hd or (heads is not None and shape[1] != heads):
        raise ValueError(f"{name} must be [n_tokens][heads][head_dim]")
    if n > 0 and (stride[2] != 1 or (stride[1] != hd and shape[1] != 1)):
        raise ValueError(f"{name}: the heads of a token must be adjacent")
    return stride[0] if n > 1 else shape[1] * hd


def kv_append(cache: KVCache, batch: KVBatch, k, v, *, rot=None, q=None, q_out=None, g_q=None, g_k=None,
              eps: float = 1e-5, pairing: str = "interleaved", stream=None):
    """Append the batch's keys and values (bf16 [n_tokens][n_kv][head_dim], rows
    a multiple of 8 elements apart) to the cache, with the norm of each head (g_q, g_k: fp32
    [head_dim] gains) and the rotation of q and k by position on the way.  rot:
    cos, sin of every position and pair, complex64 [rows][rot_dim / 2] or
    fp32 [rows][rot_dim / 2][2], rows >= 64 * max_pages.  Returns q normed and
    rotated (bf16; q_out, which may be q, or a new tensor), None without q;
    rows outside every sequence are left as they were."""
    dev, hd, n = cache.device, cache.head_dim, batch.n_tokens
    if batch.device != dev:
        raise ValueError("cache and batch are on different devices")
    if pairing not in ROPE_PAIRINGS:
        raise ValueError(f"unknown pairing {pairing!r}")
    ks = _kv_rows("k", k, n, cache.n_kv, hd, dev)
    vs = _kv_rows("v", v, n, cache.n_kv, hd, dev)
    rp, rows, dim = None, 0, 0
    if rot is not None:
        if rot.device != dev or not rot.is_contiguous() or not (
                rot.dtype is torch.complex64 and rot.dim() == 2
                or rot.dtype is torch.float32 and rot.dim() == 3 and rot.shape[2] == 2):
            raise ValueError("rot must be contiguous complex64 [rows][rot_dim / 2] or fp32 [rows][rot_dim / 2][2]")
        rp, rows, dim = rot.data_ptr(), rot.shape[0], 2 * rot.shape[1]
    for g in (g_q, g_k):
        if g is not None and not (g.dtype is torch.float32 and g.device == dev and g.is_contiguous()
                                  and g.shape == (hd,)):
            raise ValueError("g_q and g_k must be fp32 [head_dim] on the cache's device")
    r = _KVRotation(rp, rows, dim, ROPE_PAIRINGS[pairing], None if g_q is None else g_q.data_ptr(),
                    None if g_k is None else g_k.data_ptr(), eps)
    n_heads, qp, qs, qop, qos = cache.n_kv, None, 0, None, 0
    if q is not None:
        qs = _kv_rows("q", q, n, None, hd, dev)
        n_heads, qp = q.shape[1], q.data_ptr()
        if q_out is None:
            with _made_on(stream):
                q_out = torch.empty_like(q)
        qos = qs if q_out is q else _kv_rows("q_out", q_out, n, n_heads, hd, dev)
        qop = q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    sp, here = _on(stream, dev)
    _kv_call(_lib.prox_kv_append, "prox_kv_append", dev, here, cache._ref, batch._ref, k.data_ptr(), ks, v.data_ptr(),
             vs, ctypes.byref(r), n_heads, qp, qs, qop, qos, sp)
    _held_for(stream, cache, batch, k, v, q, q_out, rot, g_q, g_k)
    return q_out


def kv_workspace_bytes(cache: KVCache, batch: KVBatch, n_heads: int) -> int:
    return _lib.prox_kv_workspace_bytes(cache._ref, batch._ref, n_heads)


def alloc_kv_workspace(cache: KVCache, batch: KVBatch, n_heads: int):
    """Workspace of kv_attention for batches of this shape (n_seq, max_q, max_pages)."""
    with torch.cuda.device(cache.device):
        n = kv_workspace_bytes(cache, batch, n_heads)
    if n == 0:
        raise ValueError("invalid cache, batch or n_heads for a workspace, or bounds too large for one call")
    raw = torch.empty(n + 256, dtype=torch.uint8, device=cache.device)
    off = (-raw.data_ptr()) % 256
    return raw[off: off + n]


def kv_attention(q, cache: KVCache, batch: KVBatch, *, scale: Optional[float] = None, window: int = 0, out=None,
                 workspace=None, stream=None):
    """Causal attention of q (bf16 [n_tokens][n_heads][head_dim], rows a multiple
    of 8 elements apart, as kv_append returns it) over the cache; scale defaults to
    1 / sqrt(head_dim), window > 0 limits a row to its last `window` positions.
    Returns out, bf16 [n_tokens][n_heads][head_dim]; rows that see nothing are
    zeros, rows outside every sequence are left as they were."""
    dev, hd, n = cache.device, cache.head_dim, batch.n_tokens
    if batch.device != dev:
        raise ValueError("cache and batch are on different devices")
    if window >= 1 << 31:
        raise ValueError("window must be below 2^31")
    qs = _kv_rows("q", q, n, None, hd, dev)
    n_heads = q.shape[1]
    with _made_on(stream):
        if out is None:
            out = torch.empty_like(q)
        if workspace is None:
            workspace = alloc_kv_workspace(cache, batch, n_heads)
    os_ = _kv_rows("out", out, n, n_heads, hd, dev)
    if workspace.device != dev or not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous on the cache's device")
    sp, here = _on(stream, dev)
    _kv_call(_lib.prox_kv_attention, "prox_kv_attention", dev, here, cache._ref, batch._ref, q.data_ptr(), qs, n_heads,
             hd ** -0.5 if scale is None else scale, window, out.data_ptr(), os_, workspace.data_ptr(),
             workspace.nbytes, sp)
    _held_for(stream, cache, batch, q, out, workspace)
    return out


def kv_read(cache: KVCache, batch: KVBatch, *, dtype=torch.bfloat16, k_out=None, v_out=None, stream=None):
    """The batch's tokens back from the cache: (k, v), each [n_tokens][n_kv]
    [head_dim] in bf16 or fp32, the values that the codes stand for; zeros where
    a position or its page does not exist, and rows outside every sequence as
    they were (a new tensor's are not initialised)."""
    dev = cache.device
    if batch.device != dev:
        raise ValueError("cache and batch are on different devices")
    if dtype is not torch.bfloat16 and dtype is not torch.float32:
        raise ValueError("dtype must be bfloat16 or float32")
    shape = (batch.n_tokens, cache.n_kv, cache.head_dim)
    if k_out is None and v_out is None:
        with _made_on(stream):
            k_out, v_out = torch.empty((2,) + shape, dtype=dtype, device=dev).unbind(0)
    elif k_out is None or v_out is None:
        raise ValueError("k_out and v_out must both be given or neither")
    else:
        for t in (k_out, v_out):
            if not (t.dtype is dtype and t.device == dev and t.is_contiguous() and t.shape == shape):
                raise ValueError("k_out and v_out must be contiguous [n_tokens][n_kv][head_dim] of the dtype")
    sp, here = _on(stream, dev)
    _kv_call(_lib.prox_kv_read, "prox_kv_read", dev, here, cache._ref, batch._ref, k_out.data_ptr(), v_out.data_ptr(),
             1 if dtype is torch.float32 else 0, sp)
    _held_for(stream, cache, batch, k_out, v_out)
    return k_out, v_out


__all__ = ["KVCache", "KVBatch", "KV_KINDS", "KV_PAGE", "kv_head_pad", "kv_append", "kv_attention", "kv_read",
           "kv_workspace_bytes", "alloc_kv_workspace",
           "QWeights", "build_qweights", "qweights_bytes", "quality", "timeline_forward", "read_probe", "noalloc_scratch_bytes", "ffn_forward_noalloc", "Weights", "Proxy", "ProxError", "abi_version", "library_sha256", "proxy_bytes", "workspace_bytes",
           "build_proxy", "alloc_workspace", "ffn_forward", "LIB_PATH", "KINDS", "N_PHASES", "PHASES"]
