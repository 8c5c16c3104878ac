"""B200 (sm_100a) Reference Sliding Window Attention.

Thin Python binding over the C ABI of librswa.so (include/rswa.h).  It only
checks and marshals arguments: torch tensors supply device memory and the
current CUDA stream; every step of the attention runs in the library's CUDA
kernels.  If the library is missing or the device is not a B200 the calls
raise; nothing is computed any other way.

    attn = RSWA(L_m_cap=2592, n=128, H=10, d=128, batch=1, dtype=torch.bfloat16)
    attn.load_reference(K_ref, V_ref, ref_lens)        # [B, H, L_m_cap, d]
    o = attn.append_decode(k, v, q)                    # [B, H, d] each
    O = masked_forward(Q, K, V, L_m=..., n=128)        # [L, H, d]

Training: masked_attention (and masked_attention_varlen, over a pack of
documents) is the differentiable call; masked_backward(_varlen) is its
gradient by itself, from the O and lse of masked_forward(_varlen)(...,
return_lse=True).  Positions: Rotary turns q and k, by itself (apply) or
inside RSWA.append_decode, RSWA.prefill and masked_attention (rotary=...).
"""

from __future__ import annotations

import ctypes as C
from typing import Optional, Sequence

import numpy as np
import torch

from . import _native
from ._native import MODE_FULL, MODE_RSWA, RSWAError, check

__all__ = ["RSWA", "LayerStep", "append_decode_layers", "masked_forward", "masked_forward_varlen",
           "masked_backward", "masked_backward_varlen", "masked_attention", "masked_attention_varlen",
           "Rotary", "document_positions", "RSWAError", "MODE_RSWA", "MODE_FULL", "library_version"]

_DT = {torch.float32: _native.F32, torch.bfloat16: _native.BF16}


def library_version() -> str:
    return _native.lib().rswa_version().decode()


# The raw current-stream query avoids building a Stream object on every call.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _stream_ptr(device: torch.device) -> int:
    if _raw_stream is not None:
        return _raw_stream(device.index)
    return torch.cuda.current_stream(device).cuda_stream


def _check_tensor(name: str, t: torch.Tensor, shape, dtype, device) -> None:
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.dtype != dtype:
        raise ValueError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


_device_now = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(index: int, fn, *args) -> None:
    """fn(*args) with CUDA device `index` current; raises on its status."""
    if _device_now() == index:
        status = fn(*args)
    else:
        with torch.cuda.device(index):
            status = fn(*args)
    if status:
        check(status)


def _check_like(name: str, t: torch.Tensor, like: torch.Tensor, shape, index: int) -> None:
    """t has like's dtype, this shape, device `index` and is contiguous: in one
    pass over cached values, or by the check that names the problem."""
    if not (isinstance(t, torch.Tensor) and t.dtype is like.dtype and t.shape == shape and t.get_device() == index
            and t.is_contiguous()):
        _check_tensor(name, t, shape, like.dtype, like.device)


class RSWA:
    """Decode-side R-SWA state over caller-owned device memory.

    The K/V caches ([B, H, L_m_cap + window, d] each) and the workspace are
    torch tensors owned by this object; the library itself allocates
    nothing.  mode MODE_RSWA keeps an n-slot output ring (cache L_m + n);
    MODE_FULL keeps every output (cache L_m + T_cap), the full-attention
    baseline.
    """

    def __init__(self, L_m_cap: int, n: int, H: int, d: int, batch: int,
                 dtype: torch.dtype = torch.bfloat16, mode: int = MODE_RSWA, T_cap: int = 0,
                 device: Optional[torch.device] = None):
        if dtype not in _DT:
            raise ValueError(f"dtype {dtype} not supported (float32, bfloat16)")
        dev = torch.device(device) if device is not None else torch.device("cuda")
        if dev.type != "cuda":
            raise ValueError(f"RSWA needs a CUDA device, got {dev}")
        if dev.index is None:
            dev = torch.device("cuda", torch.cuda.current_device())
        self.device = dev
        self._dev_index = dev.index
        self._vec_shape = torch.Size((batch, H, d))
        self.L_m_cap, self.n, self.H, self.d, self.batch = L_m_cap, n, H, d, batch
        self.dtype, self.mode, self.T_cap = dtype, mode, T_cap
        self.window = n if mode == MODE_RSWA else T_cap
        L = _native.lib()
        cache_bytes = L.rswa_cache_bytes(L_m_cap, self.window, H, d, batch, _DT[dtype])
        ws_bytes = L.rswa_workspace_bytes(L_m_cap, self.window, H, d, batch)
        if cache_bytes == 0 or ws_bytes == 0:
            raise ValueError("invalid sizes for RSWA")
        self.S_cap = L_m_cap + self.window
        self.k_cache = torch.zeros((batch, H, self.S_cap, d), dtype=dtype, device=self.device)
        self.v_cache = torch.zeros((batch, H, self.S_cap, d), dtype=dtype, device=self.device)
        self.workspace = torch.empty(ws_bytes, dtype=torch.uint8, device=self.device)
        self._stream = _stream_ptr(self.device)
        h = C.c_void_p()
        with torch.cuda.device(self.device):
            check(L.rswa_init(C.byref(h), mode, L_m_cap, n, T_cap, H, d, batch, _DT[dtype],
                              self.k_cache.data_ptr(), self.v_cache.data_ptr(),
                              self.workspace.data_ptr(), ws_bytes, self._stream))
        self._h = h
        self._lib = L

    # -- plumbing
    def _sync_stream(self) -> None:
        s = _stream_ptr(self.device)
        if s != self._stream:
            check(_native.lib().rswa_set_stream(self._h, s))
            self._stream = s

    def _vec(self, name, t):
        # fast path of _check_tensor on cached values; the slow one names the problem
        if not (isinstance(t, torch.Tensor) and t.dtype == self.dtype and t.shape == self._vec_shape
                and t.get_device() == self._dev_index and t.is_contiguous()):
            _check_tensor(name, t, (self.batch, self.H, self.d), self.dtype, self.device)

    def close(self) -> None:
        if getattr(self, "_h", None):
            _native.lib().rswa_destroy(self._h)
            self._h = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

    # -- API
    def load_reference(self, K_ref: torch.Tensor, V_ref: torch.Tensor, ref_lens: Sequence[int]) -> None:
        """K_ref, V_ref: [B, H, stride, d] on the device; rows [0, ref_lens[b]) are used."""
        if K_ref.dim() != 4:
            raise ValueError("K_ref must be [B, H, stride, d]")
        stride = K_ref.shape[2]
        _check_tensor("K_ref", K_ref, (self.batch, self.H, stride, self.d), self.dtype, self.device)
        _check_tensor("V_ref", V_ref, (self.batch, self.H, stride, self.d), self.dtype, self.device)
        if len(ref_lens) != self.batch:
            raise ValueError("ref_lens must have one entry per sequence")
        lens = (C.c_int32 * self.batch)(*[int(x) for x in ref_lens])
        self._sync_stream()
        check(_native.lib().rswa_load_reference(self._h, K_ref.data_ptr(), V_ref.data_ptr(), stride, lens))

    def load_packed(self, K: torch.Tensor, V: torch.Tensor, ref_lens: Sequence[int], T0: int) -> None:
        """Cache as after load_reference + T0 appends, from the packed layout
        K, V: [B, L, H, d] (or [L, H, d] for one sequence) on the device, where
        row p of sequence b holds position p+1: the reference rows
        [0, ref_lens[b]), then output t at row ref_lens[b] + t - 1."""
        if K.dim() == 3 and self.batch == 1:
            K, V = K.unsqueeze(0), V.unsqueeze(0)
        if K.dim() != 4:
            raise ValueError("K must be [B, L, H, d]")
        L = K.shape[1]
        _check_tensor("K", K, (self.batch, L, self.H, self.d), self.dtype, self.device)
        _check_tensor("V", V, (self.batch, L, self.H, self.d), self.dtype, self.device)
        if len(ref_lens) != self.batch:
            raise ValueError("ref_lens must have one entry per sequence")
        lens = (C.c_int32 * self.batch)(*[int(x) for x in ref_lens])
        self._sync_stream()
        check(_native.lib().rswa_load_packed(self._h, K.data_ptr(), V.data_ptr(), L, lens, int(T0)))

    def load_reference_chunk(self, K: torch.Tensor, V: torch.Tensor, rows: Sequence[int]) -> None:
        """Appends rows [0, rows[b]) of K, V ([B, H, stride, d] on the device)
        to sequence b's reference, after the rows already loaded; only
        before the first output is appended."""
        if K.dim() != 4:
            raise ValueError("K must be [B, H, stride, d]")
        stride = K.shape[2]
        _check_tensor("K", K, (self.batch, self.H, stride, self.d), self.dtype, self.device)
        _check_tensor("V", V, (self.batch, self.H, stride, self.d), self.dtype, self.device)
        if len(rows) != self.batch:
            raise ValueError("rows must have one entry per sequence")
        r = (C.c_int32 * self.batch)(*[int(x) for x in rows])
        self._sync_stream()
        check(_native.lib().rswa_load_reference_chunk(self._h, K.data_ptr(), V.data_ptr(), stride, r))

    def prefill(self, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, L_m: int, scale: float = 0.0,
                out: Optional[torch.Tensor] = None, bidir_prefix: bool = False,
                rotary: Optional["Rotary"] = None) -> torch.Tensor:
        """Teacher-forced attention of one sequence (Q, K, V: [L, H, d]) with
        this handle's window, that also fills the cache as a reference load of
        rows [0, L_m) plus L - L_m appends would; decoding continues at output
        L - L_m + 1.  Batch-1 handles only.
        rotary: Q and K are turned to positions 0 .. L-1 first (into copies;
        the cache holds turned keys)."""
        if Q.dim() != 3:
            raise ValueError("Q must be [L, H, d]")
        L = Q.shape[0]
        for name, t in (("Q", Q), ("K", K), ("V", V)):
            _check_tensor(name, t, (L, self.H, self.d), self.dtype, self.device)
        O = torch.empty_like(Q) if out is None else out
        _check_tensor("out", O, (L, self.H, self.d), self.dtype, self.device)
        self._sync_stream()
        if rotary is not None:
            Q, K = rotary.apply(Q, K)
        check(_native.lib().rswa_masked_forward_fill(self._h, Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
                                                      L, int(L_m), float(scale),
                                                      _native.FLAG_BIDIR_PREFIX if bidir_prefix else 0))
        return O

    def append(self, k: torch.Tensor, v: torch.Tensor) -> None:
        self._vec("k", k)
        self._vec("v", v)
        self._sync_stream()
        check(_native.lib().rswa_append(self._h, k.data_ptr(), v.data_ptr()))

    def decode(self, q: torch.Tensor, out: Optional[torch.Tensor] = None, scale: float = 0.0) -> torch.Tensor:
        self._vec("q", q)
        o = torch.empty_like(q) if out is None else out
        self._vec("out", o)
        self._sync_stream()
        check(self._lib.rswa_decode(self._h, q.data_ptr(), o.data_ptr(), float(scale)))
        return o

    def rotate(self, rotary: "Rotary", q: torch.Tensor, k: torch.Tensor, out=None) -> tuple:
        """q, k ([B, H, d]) of the next output turned to its position, L_m[b]
        plus the outputs appended so far, read from the device-side step
        counter (so it may be captured with the append_decode that follows).
        out: a (q, k) pair, (q, k) itself for in place.  Returns the pair."""
        self._vec("q", q)
        self._vec("k", k)
        qo, ko = (torch.empty_like(q), torch.empty_like(k)) if out is None else out
        self._vec("out[0]", qo)
        self._vec("out[1]", ko)
        self._sync_stream()
        check(self._lib.rswa_rotary_step(self._h, rotary._ref, q.data_ptr(), k.data_ptr(), qo.data_ptr(),
                                         ko.data_ptr()))
        return qo, ko

    def append_decode(self, k: torch.Tensor, v: torch.Tensor, q: torch.Tensor,
                      out: Optional[torch.Tensor] = None, scale: float = 0.0,
                      rotary: Optional["Rotary"] = None) -> torch.Tensor:
        """Appends k, v and attends with q.  rotary: q and k are turned to the
        step's position first (rotate, into copies)."""
        self._vec("k", k)
        self._vec("v", v)
        self._vec("q", q)
        if rotary is not None:
            q, k = self.rotate(rotary, q, k)
        o = torch.empty_like(q) if out is None else out
        self._vec("out", o)
        self._sync_stream()
        check(self._lib.rswa_append_decode(self._h, k.data_ptr(), v.data_ptr(), q.data_ptr(),
                                           o.data_ptr(), float(scale)))
        return o

    def cache_len(self) -> list:
        out = (C.c_int32 * self.batch)()
        self._sync_stream()
        check(_native.lib().rswa_cache_len(self._h, out))
        return list(out)

    def step_count(self) -> list:
        out = (C.c_int32 * self.batch)()
        self._sync_stream()
        check(_native.lib().rswa_step_count(self._h, out))
        return list(out)

    def cache_positions(self, b: int) -> np.ndarray:
        cap = self.S_cap
        out = (C.c_int64 * cap)()
        cnt = C.c_int()
        self._sync_stream()
        check(_native.lib().rswa_cache_positions(self._h, int(b), out, cap, C.byref(cnt)))
        return np.frombuffer(out, dtype=np.int64, count=cnt.value).copy()

    def reset(self) -> None:
        self._sync_stream()
        check(_native.lib().rswa_reset(self._h))

    def check(self) -> None:
        """Raises RSWAError if a kernel flagged a device-side error."""
        self._sync_stream()
        check(_native.lib().rswa_check(self._h))


def append_decode_layers(layers: Sequence[RSWA], k: Sequence[torch.Tensor], v: Sequence[torch.Tensor],
                         q: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]] = None,
                         scale: float = 0.0) -> list:
    """One decode step of an R-layer decoder: append_decode on every layer
    handle in order (one C call, one kernel per layer).  k[r], v[r], q[r],
    out[r]: [B, H, d] tensors of layer r's handle.  Returns the outputs."""
    R = len(layers)
    if not (len(k) == len(v) == len(q) == R) or (out is not None and len(out) != R):
        raise ValueError("one k, v, q (and out) per layer")
    outs = [torch.empty_like(q[r]) for r in range(R)] if out is None else list(out)
    for r, a in enumerate(layers):
        a._vec("k", k[r])
        a._vec("v", v[r])
        a._vec("q", q[r])
        a._vec("out", outs[r])
        a._sync_stream()
    P = C.c_void_p * R
    hs = P(*[a._h.value for a in layers])
    check(_native.lib().rswa_append_decode_layers(
        hs, R, P(*[t.data_ptr() for t in k]), P(*[t.data_ptr() for t in v]), P(*[t.data_ptr() for t in q]),
        P(*[t.data_ptr() for t in outs]), float(scale)))
    return outs


class LayerStep:
    """One decode step over fixed layer handles and fixed device buffers (a
    model's per-layer k, v, q and output tensors, refilled in place every
    step): the checks and the pointer arrays are done once, so each call is
    a single C call of rswa_append_decode_layers.

    graph=True (RSWA-mode handles only) captures that call once into a CUDA
    graph and replays it on each call: the step counter lives on the device,
    so every replay is the next step.  Capture and replays do not keep the
    handles' host-side step count (read only by FULL-mode planning and the
    reference-chunk loader); step_count() reads the device counter and
    refreshes it."""

    def __init__(self, layers: Sequence[RSWA], k: Sequence[torch.Tensor], v: Sequence[torch.Tensor],
                 q: Sequence[torch.Tensor], out: Sequence[torch.Tensor], scale: float = 0.0,
                 graph: bool = False):
        R = len(layers)
        if not (len(k) == len(v) == len(q) == len(out) == R) or R < 1:
            raise ValueError("one k, v, q and out per layer")
        for r, a in enumerate(layers):
            a._vec("k", k[r])
            a._vec("v", v[r])
            a._vec("q", q[r])
            a._vec("out", out[r])
        P = C.c_void_p * R
        self._layers = list(layers)
        self._keep = (list(k), list(v), list(q), list(out))  # the tensors must outlive the step
        self._args = (P(*[a._h.value for a in layers]), R, P(*[t.data_ptr() for t in k]),
                      P(*[t.data_ptr() for t in v]), P(*[t.data_ptr() for t in q]),
                      P(*[t.data_ptr() for t in out]), float(scale))
        self._fn = _native.lib().rswa_append_decode_layers
        self._graph = None
        if graph:
            if any(a.mode != MODE_RSWA for a in layers):
                raise ValueError("graph=True needs RSWA-mode handles (FULL mode re-plans on the host)")
            dev = layers[0].device
            side = torch.cuda.Stream(dev)
            side.wait_stream(torch.cuda.current_stream(dev))
            g = torch.cuda.CUDAGraph()
            with torch.cuda.stream(side):
                with torch.cuda.graph(g, stream=side):
                    self._launch()
            torch.cuda.current_stream(dev).wait_stream(side)
            self._graph = g

    def _launch(self) -> None:
        for a in self._layers:
            a._sync_stream()
        check(self._fn(*self._args))

    def __call__(self) -> None:
        if self._graph is not None:
            self._graph.replay()
        else:
            self._launch()


def _pack_args(Q: torch.Tensor, cu_seqlens: Sequence[int], ref_lens: Sequence[int]):
    """Checks Q and the documents; -> (L, H, d, cu, refs) with the host arrays as ctypes."""
    if not Q.is_cuda:
        raise ValueError(f"Q is on {Q.device}, expected a CUDA device")
    if Q.dim() != 3:
        raise ValueError("Q must be [L, H, d]")
    L, H, d = Q.shape
    if Q.dtype not in _DT:
        raise ValueError(f"dtype {Q.dtype} not supported")
    n_docs = len(ref_lens)
    if len(cu_seqlens) != n_docs + 1 or int(cu_seqlens[-1]) != L:
        raise ValueError("cu_seqlens must have len(ref_lens) + 1 entries ending at L")
    return L, H, d, (C.c_int32 * (n_docs + 1))(*map(int, cu_seqlens)), (C.c_int32 * max(n_docs, 1))(*map(int, ref_lens))


def _forward_lse(Q, K, V, cu_seqlens, ref_lens, n, scale, out, bidir_prefix):
    L, H, d, cu, refs = _pack_args(Q, cu_seqlens, ref_lens)
    shape, index = Q.shape, Q.get_device()
    O = torch.empty_like(Q) if out is None else out
    for name, t in (("Q", Q), ("K", K), ("V", V), ("out", O)):
        _check_like(name, t, Q, shape, index)
    lse = Q.new_empty((H, L), dtype=torch.float32)
    _call(index, _native.lib().rswa_masked_forward_lse, Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
          lse.data_ptr(), cu, refs, len(ref_lens), int(n), H, d, _DT[Q.dtype], float(scale),
          _native.FLAG_BIDIR_PREFIX if bidir_prefix else 0, _stream_ptr(Q.device))
    return O, lse


def masked_forward(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, L_m: int, n: int,
                   scale: float = 0.0, out: Optional[torch.Tensor] = None,
                   bidir_prefix: bool = False, return_lse: bool = False):
    """Teacher-forced R-SWA attention.  Q, K, V, out: [L, H, d] on a B200.
    L_m = 0: no reference segment (the plain sliding window of n).
    bidir_prefix: prefix queries see every reference key (default: causal).
    return_lse: returns (O, lse) with lse float32 [H, L], the natural log of
    each row's sum of exponentials, as masked_backward takes it."""
    if Q.dim() != 3:
        raise ValueError("Q must be [L, H, d]")
    if return_lse:
        return _forward_lse(Q, K, V, (0, Q.shape[0]), (L_m,), n, scale, out, bidir_prefix)
    L, H, d = Q.shape
    if Q.dtype not in _DT:
        raise ValueError(f"dtype {Q.dtype} not supported")
    for name, t in (("K", K), ("V", V)):
        _check_tensor(name, t, (L, H, d), Q.dtype, Q.device)
    _check_tensor("Q", Q, (L, H, d), Q.dtype, Q.device)
    O = torch.empty_like(Q) if out is None else out
    _check_tensor("out", O, (L, H, d), Q.dtype, Q.device)
    with torch.cuda.device(Q.device):
        check(_native.lib().rswa_masked_forward_ex(Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
                                                   L, int(L_m), int(n), H, d, _DT[Q.dtype], float(scale),
                                                   _native.FLAG_BIDIR_PREFIX if bidir_prefix else 0,
                                                   _stream_ptr(Q.device)))
    return O


def masked_forward_varlen(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, cu_seqlens: Sequence[int],
                          ref_lens: Sequence[int], n: int, scale: float = 0.0,
                          out: Optional[torch.Tensor] = None, bidir_prefix: bool = False,
                          return_lse: bool = False):
    """Teacher-forced R-SWA attention over a pack of documents.  Q, K, V, out:
    [L, H, d] on a B200, L = cu_seqlens[-1]; document i holds rows
    cu_seqlens[i] .. cu_seqlens[i+1]-1 with ref_lens[i] reference rows and
    sees only its own keys.  return_lse: as masked_forward."""
    if return_lse:
        return _forward_lse(Q, K, V, cu_seqlens, ref_lens, n, scale, out, bidir_prefix)
    if Q.dim() != 3:
        raise ValueError("Q must be [L, H, d]")
    L, H, d = Q.shape
    if Q.dtype not in _DT:
        raise ValueError(f"dtype {Q.dtype} not supported")
    n_docs = len(ref_lens)
    if len(cu_seqlens) != n_docs + 1 or int(cu_seqlens[-1]) != L:
        raise ValueError("cu_seqlens must have len(ref_lens) + 1 entries ending at L")
    for name, t in (("Q", Q), ("K", K), ("V", V)):
        _check_tensor(name, t, (L, H, d), Q.dtype, Q.device)
    O = torch.empty_like(Q) if out is None else out
    _check_tensor("out", O, (L, H, d), Q.dtype, Q.device)
    cu = (C.c_int32 * (n_docs + 1))(*[int(x) for x in cu_seqlens])
    refs = (C.c_int32 * n_docs)(*[int(x) for x in ref_lens])
    with torch.cuda.device(Q.device):
        check(_native.lib().rswa_masked_forward_varlen(
            Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(), cu, refs, n_docs, int(n), H, d,
            _DT[Q.dtype], float(scale), _native.FLAG_BIDIR_PREFIX if bidir_prefix else 0,
            _stream_ptr(Q.device)))
    return O


def masked_backward(dO: torch.Tensor, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor,
                    lse: torch.Tensor, L_m: int, n: int, scale: float = 0.0, out=None,
                    bidir_prefix: bool = False) -> tuple:
    """Gradient of masked_forward: (dQ, dK, dV) for the gradient dO of its
    output, from its inputs and the (O, lse) it returned with return_lse=True
    (the same L_m, n, scale and bidir_prefix).  All [L, H, d], lse [H, L]
    float32.  out: three tensors to write, apart from every input.  The same
    call gives the same bits."""
    if Q.dim() != 3:
        raise ValueError("Q must be [L, H, d]")
    return masked_backward_varlen(dO, Q, K, V, O, lse, (0, Q.shape[0]), (L_m,), n, scale, out, bidir_prefix)


def masked_backward_varlen(dO: torch.Tensor, Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, O: torch.Tensor,
                           lse: torch.Tensor, cu_seqlens: Sequence[int], ref_lens: Sequence[int], n: int,
                           scale: float = 0.0, out=None, bidir_prefix: bool = False) -> tuple:
    """Gradient of masked_forward_varlen, as masked_backward: (dQ, dK, dV)."""
    if out is None:
        r = _native.binding().backward(dO, Q, K, V, O, lse, cu_seqlens, ref_lens, n, scale,
                                       _native.FLAG_BIDIR_PREFIX if bidir_prefix else 0)
        if r.__class__ is tuple:
            return r
        if r is not None:
            check(r)
    # Given results, argument types the short way leaves alone, or something that does not fit.
    L, H, d, cu, refs = _pack_args(Q, cu_seqlens, ref_lens)
    shape, index = Q.shape, Q.get_device()
    if out is None:
        grads = torch.empty_like(Q), torch.empty_like(Q), torch.empty_like(Q)
    elif len(out) == 3:
        grads = tuple(out)
    else:
        raise ValueError("out must be three tensors")
    dQ, dK, dV = grads
    for name, t in (("Q", Q), ("dO", dO), ("K", K), ("V", V), ("O", O)):
        _check_like(name, t, Q, shape, index)
    if out is not None:
        for i, t in enumerate(grads):
            _check_like(f"out[{i}]", t, Q, shape, index)
    _check_tensor("lse", lse, (H, L), torch.float32, Q.device)
    lib = _native.lib()
    dt, docs, n = _DT[Q.dtype], len(ref_lens), int(n)
    flags = _native.FLAG_BIDIR_PREFIX if bidir_prefix else 0
    ws_bytes = lib.rswa_masked_backward_workspace_bytes(cu, refs, docs, n, H, d, dt, flags)
    # 0 bytes: arguments that the call itself reports
    ws = Q.new_empty((max(ws_bytes, 16),), dtype=torch.uint8)
    _call(index, lib.rswa_masked_backward, dO.data_ptr(), Q.data_ptr(), K.data_ptr(), V.data_ptr(), O.data_ptr(),
          lse.data_ptr(), dQ.data_ptr(), dK.data_ptr(), dV.data_ptr(), cu, refs, docs, n, H, d, dt, float(scale),
          flags, ws.data_ptr(), ws_bytes, _stream_ptr(Q.device))
    return grads


class Rotary:
    """A plan of rotary positions for heads of d (64 or 128) elements.

    rotary_dim: the elements of a head that turn (even; default all of them).
    interleaved: pairs (x_2i, x_2i+1); default (x_i, x_{i + rotary_dim/2}).
    scaling, for contexts longer than trained: None, "linear" (positions
    compressed by factor), "ntk" (a larger base) or "yarn" (by parts, over the
    original_length that the model was trained on, with its magnitude
    0.1 ln(factor) + 1)."""

    _SCALINGS = {None: _native.ROTARY_PLAIN, "linear": _native.ROTARY_LINEAR, "ntk": _native.ROTARY_NTK,
                 "yarn": _native.ROTARY_YARN}

    def __init__(self, d: int, rotary_dim: Optional[int] = None, base: float = 10000.0, interleaved: bool = False,
                 scaling: Optional[str] = None, factor: float = 1.0, original_length: int = 0):
        if scaling not in self._SCALINGS:
            raise ValueError(f"scaling {scaling!r} not one of None, 'linear', 'ntk', 'yarn'")
        self.d, self.rotary_dim = int(d), int(d if rotary_dim is None else rotary_dim)
        self.interleaved = bool(interleaved)
        self._plan = _native.RotaryPlan()
        check(_native.lib().rswa_rotary_plan(C.byref(self._plan), self.d, self.rotary_dim, int(self.interleaved),
                                             float(base), self._SCALINGS[scaling], float(factor),
                                             int(original_length)))
        self.mscale = self._plan.mscale
        self._ref, self._address = C.byref(self._plan), C.addressof(self._plan)
        self._rotary = None  # the binding's function, from the first turn on: a plan alone needs no GPU build of torch
        self._made_from = (d, rotary_dim, base, interleaved, scaling, factor, original_length)

    def __reduce__(self):  # copies and pickles are made anew: the plan's address is this object's own
        return Rotary, self._made_from

    def __call__(self, Q: torch.Tensor, K: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
                 first: int = 0):
        """apply as a differentiable function of Q and K (any number of times)."""
        _check_capture(*((Q,) if K is None else (Q, K)))
        r = _Turn.apply(self, positions, first, False, *((Q,) if K is None else (Q, K)))
        return r[0] if K is None else r

    def _stride(self, name: str, t: torch.Tensor, rows: int, like: torch.Tensor, index: int) -> int:
        """Checks t ([rows, heads, d] with contiguous heads, a slice of wider
        rows or not) and returns its row stride in elements."""
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        shape, s = t.shape, t.stride()
        if len(shape) != 3 or shape[0] != rows or shape[2] != self.d:
            raise ValueError(f"{name} has shape {tuple(shape)}, expected [{rows}, heads, {self.d}]")
        if t.dtype is not like.dtype or t.get_device() != index:
            raise ValueError(f"{name} is {t.dtype} on {t.device}, expected {like.dtype} on {like.device}")
        heads = shape[1]
        if s[2] != 1 or (heads > 1 and s[1] != self.d):
            raise ValueError(f"{name} must have contiguous heads")
        return s[0] if rows > 1 else heads * self.d

    def apply(self, Q: torch.Tensor, K: Optional[torch.Tensor] = None, positions: Optional[torch.Tensor] = None,
              first: int = 0, inverse: bool = False, out=None):
        """Q (and K) [rows, heads, d] turned to their positions, in one launch
        (calling the plan itself is the differentiable form).

        positions: int32 [rows] on the device; None: first, first + 1, ...
        inverse: turned back by the same angles (the gradient).
        Rows may be slices of wider ones (a fused projection); out (Q's
        result, or the pair) may be such slices too, or the inputs
        themselves.  Returns Q's result, or the pair."""
        if out is None:
            if self._rotary is None:
                self._rotary = _native.binding().rotary
            r = self._rotary(self._address, Q, K, positions, first, inverse)
            if r.__class__ is int:
                check(r)
            if r is not None:
                return r
        # Given results, a subclass of Tensor, or something that does not fit.
        if not isinstance(Q, torch.Tensor):
            raise TypeError("Q must be a torch.Tensor")
        if not Q.is_cuda:
            raise ValueError(f"Q is on {Q.device}, expected a CUDA device")
        if Q.dtype not in _DT:
            raise ValueError(f"dtype {Q.dtype} not supported")
        rows, index = (Q.shape[0] if Q.dim() == 3 else 0), Q.get_device()
        ins = (Q,) if K is None else (Q, K)
        strides = [self._stride(name, t, rows, Q, index) for name, t in zip(("Q", "K"), ins)]
        if out is None:
            outs = tuple(torch.empty_like(t, memory_format=torch.contiguous_format) for t in ins)
        else:
            outs = (out,) if K is None else tuple(out)
        if len(outs) != len(ins):
            raise ValueError("out must hold one tensor for Q and one for K")
        args = []
        for name, t, s, o in zip(("Q", "K"), ins, strides, outs):
            so = self._stride("out of " + name, o, rows, Q, index)
            if o.shape != t.shape:
                raise ValueError(f"out of {name} has shape {tuple(o.shape)}, expected {tuple(t.shape)}")
            args += [t.data_ptr(), s, t.shape[1], o.data_ptr(), so]
        if K is None:
            args += [None, 0, 0, None, 0]
        pos = None
        if positions is not None:
            _check_tensor("positions", positions, (rows,), torch.int32, Q.device)
            pos = positions.data_ptr()
        _call(index, _native.lib().rswa_rotary_apply, self._ref, *args, pos, int(first), rows, _DT[Q.dtype],
              1 if inverse else 0, _stream_ptr(Q.device))
        return outs[0] if K is None else outs


def _check_capture(*inputs) -> None:
    """Refuses a differentiable call under stream capture whose backward pass
    would add a leaf's gradient on the default stream, which a capture may not
    reach: the backward pass would end the process.  A leaf's gradient stays
    on the stream of the first autograd graph over it for as long as any graph
    holds the leaf (a kept loss is enough)."""
    if not (inputs[0].is_cuda and torch.is_grad_enabled() and torch.cuda.is_current_stream_capturing()):
        return
    todo, seen = [t.grad_fn for t in inputs if t.grad_fn is not None], set()
    leaves = [t for t in inputs if t.grad_fn is None and t.requires_grad]
    while todo:
        node = todo.pop()
        if node in seen:
            continue
        seen.add(node)
        if hasattr(node, "variable"):
            leaves.append(node.variable)
        todo += [f for f, _ in node.next_functions if f is not None]
    if any(_native.binding().accumulates_on_default_stream(t) for t in leaves):
        raise ValueError("capture of a differentiable call while an autograd graph made on the default stream still "
                         "holds one of its leaves: drop that graph's results first, or make it on a side stream")


def document_positions(cu_seqlens: Sequence[int], device=None) -> torch.Tensor:
    """int32 positions of a pack's rows, each document from 0 on, on the
    device (copied from the host: not inside a graph capture)."""
    cu = np.asarray([int(x) for x in cu_seqlens], dtype=np.int64)
    if cu.size < 2 or cu[0] != 0 or (np.diff(cu) < 1).any():
        raise ValueError("cu_seqlens must start at 0 and increase")
    if torch.cuda.is_initialized() and torch.cuda.is_current_stream_capturing():
        raise ValueError("document_positions copies from the host: make them before the capture")
    pos = np.arange(cu[-1], dtype=np.int64) - np.repeat(cu[:-1], np.diff(cu))
    return torch.from_numpy(pos.astype(np.int32)).to(torch.device("cuda") if device is None else device)


def _grad(t: torch.Tensor) -> torch.Tensor:
    """A gradient as the kernels read it: contiguous, on a 16-byte address
    (that of a part of a concatenation may be neither)."""
    t = t.contiguous()
    return t.clone() if t.data_ptr() & 15 else t


class _Turn(torch.autograd.Function):
    @staticmethod
    def forward(ctx, rotary, positions, first, inverse, Q, K=None):
        ctx.rotary, ctx.first, ctx.inverse = rotary, first, inverse
        ctx.save_for_backward(positions)
        r = rotary.apply(Q, K, positions=positions, first=first, inverse=inverse)
        return (r,) if K is None else r

    @staticmethod
    def backward(ctx, dQ, dK=None):
        positions, = ctx.saved_tensors
        g = (_grad(dQ),) if dK is None else (_grad(dQ), _grad(dK))
        if torch.is_grad_enabled():  # create_graph: a turn is linear, and so is its gradient
            r = _Turn.apply(ctx.rotary, positions, ctx.first, not ctx.inverse, *g)
        else:
            r = ctx.rotary.apply(*g, positions=positions, first=ctx.first, inverse=not ctx.inverse)
            r = (r,) if dK is None else r
        return (None, None, None, None) + r


class _Once(torch.autograd.Function):
    """The first n tensors as they are, as functions of the others that cannot be
    differentiated.  (once_differentiable cuts the graph instead: a gradient of
    something that holds both an output and its gradient would then lack the
    second part, without a word.)"""

    @staticmethod
    def forward(ctx, n, *tensors):
        return tuple(t.view_as(t) for t in tensors[:n])

    @staticmethod
    def backward(ctx, *_):
        raise RuntimeError("masked_attention is once differentiable: its gradients (create_graph=True) have none")


class _MaskedAttention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, Q, K, V, cu_seqlens, ref_lens, n, scale, bidir_prefix, rotary, positions):
        graph = ()
        if rotary is not None:
            # What is saved of Q and K is their turned copies; an empty piece
            # of each keeps the gradients' dependence on them (and no memory).
            with torch.enable_grad():
                graph = tuple(t[:0].clone() for t in (Q, K) if t.requires_grad)
            Q, K = rotary.apply(Q, K, positions=positions)
        O, lse = _forward_lse(Q, K, V, cu_seqlens, ref_lens, n, scale, None, bidir_prefix)
        ctx.save_for_backward(Q, K, V, O, lse, positions, *graph)
        ctx.args = (cu_seqlens, ref_lens, n, scale, None, bidir_prefix)
        ctx.rotary = rotary
        return O

    @staticmethod
    def backward(ctx, dO):
        Q, K, V, O, lse, positions, *graph = ctx.saved_tensors
        with torch.no_grad():
            grads = masked_backward_varlen(_grad(dO), Q, K, V, O, lse, *ctx.args)
            if ctx.rotary is not None:
                ctx.rotary.apply(*grads[:2], positions=positions, inverse=True, out=grads[:2])
        if torch.is_grad_enabled():  # create_graph
            of = [t for t in (dO, Q, K, V, *graph) if t.requires_grad]
            if of:
                grads = _Once.apply(3, *grads, *of)
        return grads + (None,) * 7


def masked_attention(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, L_m: int, n: int, scale: float = 0.0,
                     bidir_prefix: bool = False, rotary: Optional[Rotary] = None,
                     positions: Optional[torch.Tensor] = None) -> torch.Tensor:
    """masked_forward as a differentiable function of Q, K and V, once: a
    second derivative raises, and so do forward mode and torch.func's
    transforms.  rotary: Q and K are turned first, to positions (int32
    [L] on the device; None: 0 .. L-1), and their gradients turned back."""
    if rotary is None and positions is not None:
        raise ValueError("positions without rotary")
    _check_capture(Q, K, V)
    return _MaskedAttention.apply(Q, K, V, (0, Q.shape[0]), (int(L_m),), n, scale, bidir_prefix, rotary, positions)


def masked_attention_varlen(Q: torch.Tensor, K: torch.Tensor, V: torch.Tensor, cu_seqlens: Sequence[int],
                            ref_lens: Sequence[int], n: int, scale: float = 0.0, bidir_prefix: bool = False,
                            rotary: Optional[Rotary] = None, positions: Optional[torch.Tensor] = None) -> torch.Tensor:
    """masked_forward_varlen as a differentiable function, as
    masked_attention.  rotary without positions: document_positions of the
    pack (pass them to reuse them over a model's layers or to capture)."""
    if rotary is None and positions is not None:
        raise ValueError("positions without rotary")
    if rotary is not None and positions is None:
        positions = document_positions(cu_seqlens, Q.device)
    _check_capture(Q, K, V)
    cu, refs = tuple(int(x) for x in cu_seqlens), tuple(int(x) for x in ref_lens)
    return _MaskedAttention.apply(Q, K, V, cu, refs, n, scale, bidir_prefix, rotary, positions)
