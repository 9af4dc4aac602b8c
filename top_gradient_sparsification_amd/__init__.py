"""MI355X-native error-feedback top-k gradient sparsifier.

Thin ctypes binding over ``libtgs.so`` (C ABI declared in ``include/tgs.h``).
This module only marshals arguments: every step of the three operations runs
in the library's HIP kernels.  PyTorch supplies device memory and streams.

Operations (cited by page title and section):

* ``topk_ef_step``      -- error-feedback top-k (arxivdaily listing for arXiv
  2004.05298, entries "Sparsified SGD with Memory" and "The Convergence of
  Sparsified Gradient Methods").
* ``threshold_ef_step`` -- hard-threshold sparsifier with error feedback (same
  listing, entry "Rethinking gradient sparsification as total error
  minimization").
* ``gtopk_merge``       -- the gTop-k tournament (nubint review "A Distributed
  Synchronous SGD Algorithm with Global Top-k Sparsification for Low Bandwidth
  Networks", ABSTRACT and Method).
* ``threshold_estimate`` / ``estimated_threshold_ef_step`` -- a threshold
  estimated from a sample, fed to the hard threshold on the device (arxivdaily
  listing, entry "Near-Optimal Sparse Allreduce for Distributed Deep
  Learning"; fugumt page for arXiv 2502.07634, related-paper entry "An
  Efficient Statistical-based Gradient Compression Technique for Distributed
  Training Systems").
* ``rtopk_ef_step``     -- k random entries of the top r (arxivdaily listing,
  entry "rTop-k: A Statistical Estimation Approach to Distributed SGD").

Operators of the training step around it:

* ``embedding_lookup`` / ``embedding_grad`` -- rows of an embedding table with
  scaling, and the table's dense gradient by sorted tokens.
* ``newton_schulz`` / ``muon_step`` -- a matrix orthogonalised by Newton-Schulz
  products, and the Muon update of weight matrices that takes it.
* ``layer_norm`` / ``layer_norm_grad`` -- layer norm of rows and its gradients.
* ``token_logprobs`` / ``token_logprobs_grad`` -- log probabilities of given
  tokens with entropy and top alternatives, and the logits' gradient.
* ``distillation_loss`` / ``distillation_grad`` / ``distillation_loss_and_grad``
  -- KL divergence from a teacher's top logits, its gradient, and both at once.

Gradients are reverse-mode; a tensor with a forward-mode tangent is refused.

There is no fallback: if ``libtgs.so`` is missing or cannot be loaded, every
call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from typing import NamedTuple

import numpy as np
import torch
from torch.autograd import forward_ad

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtgs.so")

TGS_OK = 0
TGS_EINVAL = -1
TGS_EWORKSPACE = -2
TGS_EHIP = -3
TGS_EDEVICE = -4

OPT_TOPK_PATH = 1
OPT_MAIN_GRID = 2

_STATUS_EXC = {TGS_EINVAL: ValueError, TGS_EWORKSPACE: MemoryError}


class TgsError(RuntimeError):
    """Raised for TGS_EHIP and TGS_EDEVICE (a bounded wait timed out or
    counts were inconsistent: the outputs of the calls since the error word was
    last read are not to be used)."""

    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


_lib = None
_lib_lock = threading.Lock()


def _load():
    global _lib
    if _lib is not None:
        return _lib
    with _lib_lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                "libtgs.so not found at %s; build it with "
                "`python -m top_gradient_sparsification_amd.build`" % LIB_PATH)
        # torch is imported first, so the library binds to torch's HIP runtime
        # (same soname) and torch streams are valid handles for it.
        lib = ctypes.CDLL(LIB_PATH)
        i64, i32, vp, sz = ctypes.c_int64, ctypes.c_int32, ctypes.c_void_p, ctypes.c_size_t
        lib.tgs_topk_workspace_bytes.argtypes = [i64, i64]
        lib.tgs_topk_workspace_bytes.restype = sz
        lib.tgs_topk_ef_step.argtypes = [vp, vp, i64, i64, vp, vp, vp, sz, vp]
        lib.tgs_topk_ef_step.restype = i32
        lib.tgs_topk_segmented_workspace_bytes.argtypes = [i32, vp, vp]
        lib.tgs_topk_segmented_workspace_bytes.restype = sz
        lib.tgs_topk_ef_step_segmented.argtypes = [vp, vp, i32, vp, vp, vp, vp, vp, sz, vp]
        lib.tgs_topk_ef_step_segmented.restype = i32
        lib.tgs_threshold_workspace_bytes.argtypes = [i64]
        lib.tgs_threshold_workspace_bytes.restype = sz
        lib.tgs_threshold_ef_step.argtypes = [vp, vp, i64, ctypes.c_float, vp, vp, i64, vp, vp, sz, vp]
        lib.tgs_threshold_ef_step.restype = i32
        lib.tgs_gtopk_workspace_bytes.argtypes = [i32, i64, i64]
        lib.tgs_gtopk_workspace_bytes.restype = sz
        lib.tgs_gtopk_merge.argtypes = [vp, vp, i32, i64, i64, vp, vp, vp, vp, sz, vp]
        lib.tgs_gtopk_merge.restype = i32
        lib.tgs_check_device_error.argtypes = [vp, vp]
        lib.tgs_check_device_error.restype = i32
        lib.tgs_workspace_init.argtypes = [vp, sz, vp]
        lib.tgs_workspace_init.restype = i32
        lib.tgs_threshold_estimate_workspace_bytes.argtypes = [i64]
        lib.tgs_threshold_estimate_workspace_bytes.restype = sz
        lib.tgs_threshold_estimate.argtypes = [vp, vp, i64, vp, i64, i64, vp, vp, sz, vp]
        lib.tgs_threshold_estimate.restype = i32
        lib.tgs_threshold_ef_step_dev.argtypes = [vp, vp, i64, vp, vp, vp, i64, vp, vp, sz, vp]
        lib.tgs_threshold_ef_step_dev.restype = i32
        u64 = ctypes.c_uint64
        lib.tgs_rtopk_workspace_bytes.argtypes = [i64, i64, i64]
        lib.tgs_rtopk_workspace_bytes.restype = sz
        lib.tgs_rtopk_ef_step.argtypes = [vp, vp, i64, i64, i64, u64, u64, vp, vp, vp, sz, vp]
        lib.tgs_rtopk_ef_step.restype = i32
        f32 = ctypes.c_float
        lib.tgs_embedding_lookup_workspace_bytes.argtypes = [i64]
        lib.tgs_embedding_lookup_workspace_bytes.restype = sz
        lib.tgs_embedding_lookup.argtypes = [vp, i32, i64, vp, i32, i64, i64, f32, vp, i32, vp, sz, vp]
        lib.tgs_embedding_lookup.restype = i32
        lib.tgs_embedding_grad_workspace_bytes.argtypes = [i64, i64, i64, i32, i32]
        lib.tgs_embedding_grad_workspace_bytes.restype = sz
        lib.tgs_embedding_grad.argtypes = [vp, i32, i64, vp, i32, i64, i64, f32, vp, i32, i32, vp, sz, vp]
        lib.tgs_embedding_grad.restype = i32
        lib.tgs_newton_schulz_workspace_bytes.argtypes = [i64, i64, i64, i32]
        lib.tgs_newton_schulz_workspace_bytes.restype = sz
        lib.tgs_newton_schulz.argtypes = [vp, i32, i64, i64, i64, i32, f32, f32, f32, f32, vp, vp, sz, vp]
        lib.tgs_newton_schulz.restype = i32
        lib.tgs_muon_workspace_bytes.argtypes = [i64, i64, i64, i32]
        lib.tgs_muon_workspace_bytes.restype = sz
        lib.tgs_muon_step.argtypes = [vp, i32, vp, i32, vp, i64, i64, i64, f32, f32, i32, f32, i32, f32, f32, f32, f32,
                                      vp, sz, vp]
        lib.tgs_muon_step.restype = i32
        lib.tgs_layer_norm.argtypes = [vp, i32, i64, i64, vp, vp, i32, f32, vp, i32, vp, vp, vp]
        lib.tgs_layer_norm.restype = i32
        lib.tgs_layer_norm_grad_workspace_bytes.argtypes = [i64, i64]
        lib.tgs_layer_norm_grad_workspace_bytes.restype = sz
        lib.tgs_layer_norm_grad.argtypes = [vp, i32, vp, i32, i64, i64, vp, vp, vp, i32, vp, vp, vp, i32, vp, sz, vp]
        lib.tgs_layer_norm_grad.restype = i32
        lib.tgs_token_logprobs_workspace_bytes.argtypes = [i64, i64, i32, i32]
        lib.tgs_token_logprobs_workspace_bytes.restype = sz
        lib.tgs_token_logprobs.argtypes = [vp, i32, i64, i64, i64, vp, i32, f32, vp, vp, vp, i32, vp, vp, vp, sz, vp]
        lib.tgs_token_logprobs.restype = i32
        lib.tgs_token_logprobs_grad.argtypes = [vp, i32, i64, i64, i64, vp, i32, f32, vp, vp, vp, vp, vp, i64, vp, sz,
                                                vp]
        lib.tgs_token_logprobs_grad.restype = i32
        lib.tgs_distillation_workspace_bytes.argtypes = [i64, i64, i32]
        lib.tgs_distillation_workspace_bytes.restype = sz
        slots = [vp, i32, i64, i64, i64, vp, i32, vp, i32, i64, f32]
        lib.tgs_distillation_loss.argtypes = [*slots, vp, vp, vp, sz, vp]
        lib.tgs_distillation_loss.restype = i32
        lib.tgs_distillation_grad.argtypes = [*slots, vp, vp, vp, i64, vp, sz, vp]
        lib.tgs_distillation_grad.restype = i32
        lib.tgs_distillation_loss_and_grad.argtypes = [*slots, vp, vp, vp, i64, vp, sz, vp]
        lib.tgs_distillation_loss_and_grad.restype = i32
        lib.tgs_status_string.argtypes = [i32]
        lib.tgs_status_string.restype = ctypes.c_char_p
        lib.tgs_last_error.argtypes = []
        lib.tgs_last_error.restype = ctypes.c_char_p
        lib.tgs_set_option.argtypes = [i32, i64]
        lib.tgs_set_option.restype = i32
        lib.tgs_profile_next_call.argtypes = [vp, vp]
        lib.tgs_profile_next_call.restype = i32
        lib.tgs_profile_elapsed_ms.argtypes = [vp, vp, ctypes.POINTER(ctypes.c_float)]
        lib.tgs_profile_elapsed_ms.restype = i32
        _lib = lib
    return _lib


def library():
    """The loaded ctypes library (raises if it is missing)."""
    return _load()


def _check(status: int, what: str):
    if status == TGS_OK:
        return
    lib = _load()
    msg = "%s: %s (%s)" % (what, lib.tgs_status_string(status).decode(), lib.tgs_last_error().decode())
    raise _STATUS_EXC.get(status, TgsError)(msg) if status in _STATUS_EXC else TgsError(status, msg)


def _stream_handle(device) -> int:
    index = (device if isinstance(device, torch.device) else torch.device(device)).index
    # the handle alone: a torch.cuda.Stream object costs 2 us a call
    return torch._C._cuda_getCurrentRawStream(torch.cuda.current_device() if index is None else index)


def _ptr(t) -> int | None:
    return t.data_ptr() if t is not None and t.numel() > 0 else None


def _full_device(device) -> torch.device:
    """``device`` with its index filled in ("cuda" -> the current device)."""
    dev = torch.device(device)
    if dev.type == "cuda" and dev.index is None:
        dev = torch.device("cuda", torch.cuda.current_device())
    return dev


def _require(t, dtype, name, device=None, min_numel=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if not t.is_cuda:
        raise TypeError("%s must be a GPU tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if min_numel is not None and t.numel() < min_numel:
        raise ValueError("%s holds %d entries, needs %d" % (name, t.numel(), min_numel))


def _require_ws(ws, dev):
    """A workspace of the caller's: kernels write to it, so host memory or another device's is refused."""
    if not isinstance(ws, torch.Tensor):
        raise TypeError("ws must be a torch.Tensor")
    if ws.device != dev:
        raise ValueError("ws is on %s, expected %s" % (ws.device, dev))
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")


# --------------------------------------------------------------- workspaces --
class _Workspaces(threading.local):
    """Each thread's own: a call enqueues a sequence of launches with the
    interpreter's lock let go, so what two threads enqueue on one stream can
    stand there mixed, and stream order alone does not keep them apart."""

    def __init__(self):
        self.buffers: dict = {}


_ws_cache = _Workspaces()


_HEADER_BYTES = 32768  # of a workspace; the rest is scratch


def workspace(kind: str, nbytes: int, device) -> torch.Tensor:
    """A zero-initialised (hence ready) uint8 device buffer of at least
    ``nbytes``, cached per (thread, device, current stream, kind).  Calls that
    share it come from one thread and are ordered on that stream.

    While the current stream is being captured it is a buffer of its own, of
    the graph's memory, its header cleared by the graph: a cached one may be
    replaced by a larger one, and the graph would write to freed memory."""
    dev = torch.device(device)
    if torch.cuda.is_current_stream_capturing():
        buf = torch.empty(max(nbytes, 256), dtype=torch.uint8, device=dev)
        buf[:_HEADER_BYTES].zero_()
        return buf
    key = (dev.index, _stream_handle(dev), kind)
    buf = _ws_cache.buffers.get(key)
    if buf is None or buf.numel() < nbytes:
        buf = torch.zeros(max(nbytes, 256), dtype=torch.uint8, device=dev)
        _ws_cache.buffers[key] = buf
    return buf


def _scratch(kind: str, nbytes: int, dev: torch.device, stream: int) -> torch.Tensor:
    """``workspace`` for a tensor's device and its current stream."""
    buf = _ws_cache.buffers.get((dev.index, stream, kind))
    if buf is None or buf.numel() < nbytes or torch.cuda.is_current_stream_capturing():
        return workspace(kind, nbytes, dev)
    return buf


# --------------------------------------------------------------- operations --
def topk_workspace_bytes(n: int, k: int) -> int:
    return int(_load().tgs_topk_workspace_bytes(n, k))


def topk_ef_step(grad: torch.Tensor, residual: torch.Tensor, k: int, out_idx=None, out_val=None,
                 ws: torch.Tensor | None = None):
    """One error-feedback top-k step on the GPU.

    ``residual`` (float32, same length as ``grad``) is updated in place to
    ``acc`` with the selected entries zeroed, where ``acc = residual + grad``.
    Returns ``(idx int32[k], val float32[k])`` in (|acc| desc, index asc) order.
    """
    _require(grad, torch.float32, "grad")
    _require(residual, torch.float32, "residual")
    n = grad.numel()
    if residual.numel() != n or residual.device != grad.device:
        raise ValueError("grad and residual must have the same length and device")
    k = int(k)
    dev = grad.device
    if out_idx is None:
        out_idx = torch.empty(k, dtype=torch.int32, device=dev)
    if out_val is None:
        out_val = torch.empty(k, dtype=torch.float32, device=dev)
    _require(out_idx, torch.int32, "out_idx")
    _require(out_val, torch.float32, "out_val")
    if out_idx.numel() < k or out_val.numel() < k:
        raise ValueError("outputs hold fewer than k entries")
    lib = _load()
    need = lib.tgs_topk_workspace_bytes(n, k)
    if need == 0:
        raise ValueError("invalid sizes n=%d k=%d" % (n, k))
    if ws is None:
        ws = workspace("topk", need, dev)
    else:
        _require_ws(ws, dev)
    st = lib.tgs_topk_ef_step(_ptr(grad), _ptr(residual), n, k, _ptr(out_idx), _ptr(out_val), ws.data_ptr(),
                              ws.numel(), _stream_handle(dev))
    _check(st, "tgs_topk_ef_step")
    return out_idx[:k], out_val[:k]


def workspace_init(ws: torch.Tensor, stream=None):
    """Makes ``ws`` ready for any operation (a kernel zero-fills its header on
    the current stream): for workspaces not allocated zero-filled, and after a
    TGS_EDEVICE report."""
    if not isinstance(ws, torch.Tensor) or not ws.is_cuda:
        raise TypeError("ws must be a GPU tensor")
    st = stream.cuda_stream if stream is not None else _stream_handle(ws.device)
    _check(_load().tgs_workspace_init(ws.data_ptr(), ws.numel() * ws.element_size(), st), "tgs_workspace_init")


def error_word(ws: torch.Tensor) -> torch.Tensor:
    """The device error word of workspace ``ws`` as a one-element int32 device
    tensor (a view: no copy, no wait).  Nonzero means a kernel flagged a
    problem since the word was last cleared by ``check_device_error``."""
    return ws[:4].view(torch.int32)


class TopkStep:
    """A prepared top-k step for repeated calls on tensors of one shape.

    Holds the outputs, the workspace and the stream, so a call costs one C-ABI
    call plus a few attribute checks: for training loops that sparsify the same
    buffer every iteration.  The library still validates every call.  Calls
    are asynchronous: ``check()`` (or ``error`` for a device-side flag) reports
    whether a kernel flagged a problem."""

    def __init__(self, n: int, k: int, device="cuda", stream=None):
        lib = _load()
        self.n, self.k = int(n), int(k)
        self.device = _full_device(device)
        need = lib.tgs_topk_workspace_bytes(self.n, self.k)
        if need == 0:
            raise ValueError("invalid sizes n=%d k=%d" % (n, k))
        self.ws = torch.zeros(need, dtype=torch.uint8, device=self.device)
        self.out_idx = torch.empty(self.k, dtype=torch.int32, device=self.device)
        self.out_val = torch.empty(self.k, dtype=torch.float32, device=self.device)
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        self._fn = lib.tgs_topk_ef_step
        self._args = (self.out_idx.data_ptr() if self.k else None, self.out_val.data_ptr() if self.k else None,
                      self.ws.data_ptr(), self.ws.numel(), self.stream.cuda_stream)

    def __call__(self, grad: torch.Tensor, residual: torch.Tensor):
        for t, name in ((grad, "grad"), (residual, "residual")):
            if (t.dtype != torch.float32 or t.device != self.device or t.numel() != self.n
                    or not t.is_contiguous()):
                _require(t, torch.float32, name, self.device)
                raise ValueError("this step is prepared for n=%d, %s holds %d" % (self.n, name, t.numel()))
        oi, ov, wp, wn, st = self._args
        status = self._fn(grad.data_ptr(), residual.data_ptr(), self.n, self.k, oi, ov, wp, wn, st)
        if status:
            _check(status, "tgs_topk_ef_step")
        return self.out_idx, self.out_val

    @property
    def error(self) -> torch.Tensor:
        """The workspace's device error word (int32 device tensor, no wait)."""
        return error_word(self.ws)

    def check(self):
        """Waits for the stream and raises if a kernel flagged a problem."""
        _check(_load().tgs_check_device_error(self.ws.data_ptr(), self.stream.cuda_stream), "tgs_topk_ef_step")


def _segment_table(offsets, ks):
    """(nseg, int64 offsets[nseg+1], int64 ks[nseg]) as contiguous host arrays."""
    offs = np.ascontiguousarray(np.asarray(offsets, dtype=np.int64))
    kk = np.ascontiguousarray(np.asarray(ks, dtype=np.int64))
    if offs.ndim != 1 or kk.ndim != 1 or offs.size != kk.size + 1:
        raise ValueError("offsets must have one entry more than ks")
    return int(kk.size), offs, kk


def topk_segmented_workspace_bytes(offsets, ks) -> int:
    nseg, offs, kk = _segment_table(offsets, ks)
    return int(_load().tgs_topk_segmented_workspace_bytes(nseg, offs.ctypes.data, kk.ctypes.data))


def topk_ef_step_segmented(grad: torch.Tensor, residual: torch.Tensor, offsets, ks, out_idx=None, out_val=None,
                           ws: torch.Tensor | None = None):
    """Layer-wise error-feedback top-k: segment s = [offsets[s], offsets[s+1])
    of ``grad``/``residual`` gets the top-k step with k = ks[s], in one call.

    Returns ``(idx int32[sum ks], val float32[sum ks])``: segment s's pairs
    start at ``sum(ks[:s])``, with indices relative to the segment's start."""
    _require(grad, torch.float32, "grad")
    _require(residual, torch.float32, "residual")
    nseg, offs, kk = _segment_table(offsets, ks)
    n = grad.numel()
    if residual.numel() != n or residual.device != grad.device:
        raise ValueError("grad and residual must have the same length and device")
    if nseg and int(offs[-1]) != n:
        raise ValueError("offsets[-1] must equal the vector length")
    total = int(kk.sum()) if nseg else 0
    dev = grad.device
    if out_idx is None:
        out_idx = torch.empty(total, dtype=torch.int32, device=dev)
    if out_val is None:
        out_val = torch.empty(total, dtype=torch.float32, device=dev)
    _require(out_idx, torch.int32, "out_idx")
    _require(out_val, torch.float32, "out_val")
    if out_idx.numel() < total or out_val.numel() < total:
        raise ValueError("outputs hold fewer than sum(ks) entries")
    lib = _load()
    need = lib.tgs_topk_segmented_workspace_bytes(nseg, offs.ctypes.data, kk.ctypes.data)
    if need == 0:
        raise ValueError("invalid segment table")
    if ws is None:
        ws = workspace("topk", need, dev)
    else:
        _require_ws(ws, dev)
    st = lib.tgs_topk_ef_step_segmented(_ptr(grad), _ptr(residual), nseg, offs.ctypes.data, kk.ctypes.data,
                                        _ptr(out_idx), _ptr(out_val), ws.data_ptr(), ws.numel(), _stream_handle(dev))
    _check(st, "tgs_topk_ef_step_segmented")
    return out_idx[:total], out_val[:total]


class TopkSegments:
    """A prepared layer-wise top-k step (fixed segment table) for repeated
    calls: holds the host table, the outputs, the workspace and the stream."""

    def __init__(self, offsets, ks, device="cuda", stream=None):
        lib = _load()
        self.nseg, self.offsets, self.ks = _segment_table(offsets, ks)
        self.n = int(self.offsets[-1]) if self.nseg else 0
        self.total = int(self.ks.sum()) if self.nseg else 0
        self.device = _full_device(device)
        need = lib.tgs_topk_segmented_workspace_bytes(self.nseg, self.offsets.ctypes.data, self.ks.ctypes.data)
        if need == 0:
            raise ValueError("invalid segment table")
        self.ws = torch.zeros(need, dtype=torch.uint8, device=self.device)
        self.out_idx = torch.empty(max(self.total, 1), dtype=torch.int32, device=self.device)
        self.out_val = torch.empty(max(self.total, 1), dtype=torch.float32, device=self.device)
        self.stream = stream if stream is not None else torch.cuda.current_stream(self.device)
        self._fn = lib.tgs_topk_ef_step_segmented
        self._args = (self.nseg, self.offsets.ctypes.data, self.ks.ctypes.data, self.out_idx.data_ptr(),
                      self.out_val.data_ptr(), self.ws.data_ptr(), self.ws.numel(), self.stream.cuda_stream)

    def __call__(self, grad: torch.Tensor, residual: torch.Tensor):
        for t, name in ((grad, "grad"), (residual, "residual")):
            if (t.dtype != torch.float32 or t.device != self.device or t.numel() != self.n
                    or not t.is_contiguous()):
                _require(t, torch.float32, name, self.device)
                raise ValueError("this call is prepared for n=%d, %s holds %d" % (self.n, name, t.numel()))
        ns, op, kp, oi, ov, wp, wn, st = self._args
        status = self._fn(grad.data_ptr(), residual.data_ptr(), ns, op, kp, oi, ov, wp, wn, st)
        if status:
            _check(status, "tgs_topk_ef_step_segmented")
        return self.out_idx[:self.total], self.out_val[:self.total]

    @property
    def error(self) -> torch.Tensor:
        """The workspace's device error word (int32 device tensor, no wait)."""
        return error_word(self.ws)

    def check(self):
        """Waits for the stream and raises if a kernel flagged a problem."""
        _check(_load().tgs_check_device_error(self.ws.data_ptr(), self.stream.cuda_stream),
               "tgs_topk_ef_step_segmented")


def threshold_workspace_bytes(n: int) -> int:
    return int(_load().tgs_threshold_workspace_bytes(n))


def threshold_ef_step(grad: torch.Tensor, residual: torch.Tensor, lam: float, capacity: int,
                      out_idx=None, out_val=None, count=None, ws: torch.Tensor | None = None):
    """One hard-threshold step on the GPU.

    Returns ``(idx int32[capacity], val float32[capacity], count int64[1])``:
    the first ``min(count, capacity)`` entries of idx/val are the qualifying
    entries in ascending index order; ``count`` (a device tensor) is the total
    number of qualifying entries.
    """
    _require(grad, torch.float32, "grad")
    _require(residual, torch.float32, "residual")
    n = grad.numel()
    if residual.numel() != n or residual.device != grad.device:
        raise ValueError("grad and residual must have the same length and device")
    dev = grad.device
    capacity = int(capacity)
    if capacity < 0:
        raise ValueError("capacity must be >= 0")
    if out_idx is None:
        out_idx = torch.empty(capacity, dtype=torch.int32, device=dev)
    if out_val is None:
        out_val = torch.empty(capacity, dtype=torch.float32, device=dev)
    if count is None:
        count = torch.empty(1, dtype=torch.int64, device=dev)
    _require(out_idx, torch.int32, "out_idx", dev, capacity)
    _require(out_val, torch.float32, "out_val", dev, capacity)
    _require(count, torch.int64, "count", dev, 1)
    lib = _load()
    need = lib.tgs_threshold_workspace_bytes(n)
    if need == 0:
        raise ValueError("invalid size n=%d" % n)
    if ws is None:
        ws = workspace("threshold", need, dev)
    else:
        _require_ws(ws, dev)
    st = lib.tgs_threshold_ef_step(_ptr(grad), _ptr(residual), n, ctypes.c_float(lam), _ptr(out_idx),
                                   _ptr(out_val), capacity, count.data_ptr(), ws.data_ptr(), ws.numel(),
                                   _stream_handle(dev))
    _check(st, "tgs_threshold_ef_step")
    return out_idx, out_val, count


def threshold_estimate_workspace_bytes(m: int) -> int:
    return int(_load().tgs_threshold_estimate_workspace_bytes(m))


def threshold_estimate(grad: torch.Tensor, residual: torch.Tensor, sample_idx: torch.Tensor, q: int,
                       d_lambda: torch.Tensor | None = None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """The q-th largest |residual + grad| over the positions ``sample_idx``
    (int32 device tensor), as a one-element float32 device tensor (no host
    round trip).  grad and residual are only read."""
    _require(grad, torch.float32, "grad")
    dev = grad.device
    _require(residual, torch.float32, "residual", dev, grad.numel())
    _require(sample_idx, torch.int32, "sample_idx", dev)
    n, m = grad.numel(), sample_idx.numel()
    if residual.numel() != n:
        raise ValueError("grad and residual must have the same length")
    if d_lambda is None:
        d_lambda = torch.empty(1, dtype=torch.float32, device=dev)
    _require(d_lambda, torch.float32, "d_lambda", dev, 1)
    lib = _load()
    need = lib.tgs_threshold_estimate_workspace_bytes(m)
    if need == 0:
        raise ValueError("invalid sample count m=%d" % m)
    if ws is None:
        ws = workspace("estimate", need, dev)
    else:
        _require_ws(ws, dev)
    st = lib.tgs_threshold_estimate(_ptr(grad), _ptr(residual), n, _ptr(sample_idx), m, int(q), d_lambda.data_ptr(),
                                    ws.data_ptr(), ws.numel(), _stream_handle(dev))
    _check(st, "tgs_threshold_estimate")
    return d_lambda


def threshold_ef_step_dev(grad: torch.Tensor, residual: torch.Tensor, d_lambda: torch.Tensor, capacity: int,
                          out_idx=None, out_val=None, count=None, ws: torch.Tensor | None = None):
    """``threshold_ef_step`` with the threshold in device memory (a
    one-element float32 tensor, read when the kernels run)."""
    _require(grad, torch.float32, "grad")
    dev = grad.device
    _require(residual, torch.float32, "residual", dev)
    _require(d_lambda, torch.float32, "d_lambda", dev, 1)
    n = grad.numel()
    if residual.numel() != n:
        raise ValueError("grad and residual must have the same length")
    capacity = int(capacity)
    if capacity < 0:
        raise ValueError("capacity must be >= 0")
    if out_idx is None:
        out_idx = torch.empty(capacity, dtype=torch.int32, device=dev)
    if out_val is None:
        out_val = torch.empty(capacity, dtype=torch.float32, device=dev)
    if count is None:
        count = torch.empty(1, dtype=torch.int64, device=dev)
    _require(out_idx, torch.int32, "out_idx", dev, capacity)
    _require(out_val, torch.float32, "out_val", dev, capacity)
    _require(count, torch.int64, "count", dev, 1)
    lib = _load()
    need = lib.tgs_threshold_workspace_bytes(n)
    if need == 0:
        raise ValueError("invalid size n=%d" % n)
    if ws is None:
        ws = workspace("threshold", need, dev)
    else:
        _require_ws(ws, dev)
    st = lib.tgs_threshold_ef_step_dev(_ptr(grad), _ptr(residual), n, d_lambda.data_ptr(), _ptr(out_idx),
                                       _ptr(out_val), capacity, count.data_ptr(), ws.data_ptr(), ws.numel(),
                                       _stream_handle(dev))
    _check(st, "tgs_threshold_ef_step_dev")
    return out_idx, out_val, count


def estimated_threshold_ef_step(grad: torch.Tensor, residual: torch.Tensor, sample_idx: torch.Tensor, q: int,
                                capacity: int, out_idx=None, out_val=None, count=None, d_lambda=None,
                                ws: torch.Tensor | None = None):
    """The sampled estimate, then the hard-threshold step with it, both on
    the current stream with no host round trip.  Returns ``(idx, val, count,
    d_lambda)`` (device tensors).  ``ws``, if given, must be large enough for
    both calls."""
    n, m = grad.numel(), sample_idx.numel()
    if ws is None:
        need = max(threshold_estimate_workspace_bytes(m), threshold_workspace_bytes(n))
        ws = workspace("threshold", need, grad.device)
    else:
        _require_ws(ws, grad.device)
    d_lambda = threshold_estimate(grad, residual, sample_idx, q, d_lambda=d_lambda, ws=ws)
    idx, val, cnt = threshold_ef_step_dev(grad, residual, d_lambda, capacity, out_idx=out_idx, out_val=out_val,
                                          count=count, ws=ws)
    return idx, val, cnt, d_lambda


def rtopk_workspace_bytes(n: int, r: int, k: int) -> int:
    return int(_load().tgs_rtopk_workspace_bytes(n, r, k))


def rtopk_ef_step(grad: torch.Tensor, residual: torch.Tensor, r: int, k: int, seed: int, step: int,
                  out_idx=None, out_val=None, ws: torch.Tensor | None = None):
    """One rTop-k step: k entries drawn at random (Philox4x32-10 keyed by
    ``seed``, counter by entry index and ``step``) from the top r of
    |residual + grad|.  ``residual`` is updated in place.  Returns ``(idx
    int32[k], val float32[k])`` in (|acc| desc, index asc) order."""
    _require(grad, torch.float32, "grad")
    dev = grad.device
    _require(residual, torch.float32, "residual", dev)
    n = grad.numel()
    if residual.numel() != n:
        raise ValueError("grad and residual must have the same length")
    r, k = int(r), int(k)
    if out_idx is None:
        out_idx = torch.empty(k, dtype=torch.int32, device=dev)
    if out_val is None:
        out_val = torch.empty(k, dtype=torch.float32, device=dev)
    _require(out_idx, torch.int32, "out_idx", dev, k)
    _require(out_val, torch.float32, "out_val", dev, k)
    lib = _load()
    need = lib.tgs_rtopk_workspace_bytes(n, r, k)
    if need == 0:
        raise ValueError("invalid sizes n=%d r=%d k=%d" % (n, r, k))
    if ws is None:
        ws = workspace("rtopk", need, dev)
    else:
        _require_ws(ws, dev)
    st = lib.tgs_rtopk_ef_step(_ptr(grad), _ptr(residual), n, r, k, int(seed) & (2**64 - 1), int(step) & (2**64 - 1),
                               _ptr(out_idx), _ptr(out_val), ws.data_ptr(), ws.numel(), _stream_handle(dev))
    _check(st, "tgs_rtopk_ef_step")
    return out_idx[:k], out_val[:k]


def gtopk_workspace_bytes(P: int, k: int, n: int) -> int:
    return int(_load().tgs_gtopk_workspace_bytes(P, k, n))


def gtopk_merge(idx: torch.Tensor, val: torch.Tensor, n: int, ws: torch.Tensor | None = None,
                check: bool = False):
    """gTop-k tournament of the P rows of ``idx``/``val`` (shape [P, k]).

    Returns ``(gidx int32[k], gval float32[k], mask uint8[P, k])``,
    asynchronously.  With ``check`` the call also waits for the device and
    raises ValueError if a row broke the index precondition (distinct indices
    inside [0, n)); otherwise ``check_device_error(ws)`` reports it later."""
    _require(idx, torch.int32, "idx")
    _require(val, torch.float32, "val")
    if idx.dim() != 2 or idx.shape != val.shape:
        raise ValueError("idx and val must both have shape [P, k]")
    P, k = idx.shape
    dev = idx.device
    out_idx = torch.empty(k, dtype=torch.int32, device=dev)
    out_val = torch.empty(k, dtype=torch.float32, device=dev)
    mask = torch.empty((P, k), dtype=torch.uint8, device=dev)
    lib = _load()
    need = lib.tgs_gtopk_workspace_bytes(P, k, n)
    if need == 0:
        raise ValueError("invalid sizes P=%d k=%d n=%d" % (P, k, n))
    if ws is None:
        ws = workspace("gtopk", need, dev)
    else:
        _require_ws(ws, dev)
    st = lib.tgs_gtopk_merge(_ptr(idx), _ptr(val), P, k, n, _ptr(out_idx), _ptr(out_val), _ptr(mask),
                             ws.data_ptr(), ws.numel(), _stream_handle(dev))
    _check(st, "tgs_gtopk_merge")
    if check:
        _check(lib.tgs_check_device_error(ws.data_ptr(), _stream_handle(dev)), "tgs_gtopk_merge (device)")
    return out_idx, out_val, mask


# ------------------------------------ operators of the training step around --
_DTYPES = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2, torch.int32: 3, torch.int64: 4}
_FLOATS = (torch.float32, torch.bfloat16, torch.float16)
_TOKENS = (torch.int32, torch.int64)


def _no_tangent(t, name):
    """Refuses a dual tensor: the result of a call that autograd cannot see has no tangent, which reads as a zero one."""
    if forward_ad.unpack_dual(t).tangent is not None:
        raise NotImplementedError("%s has a tangent, and the call no forward-mode derivative" % name)


def _require_any(t, dtypes, name, device=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if forward_ad._current_level >= 0:  # a level of forward mode is open
        _no_tangent(t, name)
    if t.dtype not in dtypes:
        raise TypeError("%s must be one of %s, got %s" % (name, ", ".join(map(str, dtypes)), t.dtype))
    if not t.is_cuda:
        raise TypeError("%s must be a GPU tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)


def _differentiable(name, out) -> bool:
    """Whether a graph is to be kept of a call on a tensor that requires a gradient; ``out`` takes none."""
    if not torch.is_grad_enabled():
        return False
    if out is not None:
        raise RuntimeError("%s requires a gradient, which a call with out= has not" % name)
    return True


def _written(t):
    """Tells autograd, which cannot see it, that a call has overwritten ``t``."""
    if not t.is_inference():
        torch.autograd.graph.increment_version(t)


class _Lookup(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, table, scale, out_dtype, ws):
        ctx.save_for_backward(tokens)
        ctx.rows, ctx.scale, ctx.dtype = table.shape[0], scale, table.dtype
        return embedding_lookup(tokens, table, scale, out_dtype, ws=ws)

    @staticmethod
    def backward(ctx, grad):
        (tokens,) = ctx.saved_tensors
        return None, embedding_grad(tokens, grad.contiguous(), ctx.rows, ctx.scale, ctx.dtype), None, None, None


class _LookupGrad(torch.autograd.Function):
    @staticmethod
    def forward(ctx, tokens, grad, num_rows, scale, out_dtype, ws):
        ctx.save_for_backward(tokens)
        ctx.scale, ctx.dtype = scale, grad.dtype
        return embedding_grad(tokens, grad, num_rows, scale, out_dtype, ws=ws)

    @staticmethod
    def backward(ctx, grad):
        (tokens,) = ctx.saved_tensors
        return None, embedding_lookup(tokens, grad.contiguous(), ctx.scale, ctx.dtype), None, None, None, None


class _NewtonSchulz(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, steps, coefficients, eps, ws):
        return newton_schulz(x, steps, coefficients, eps, ws=ws)

    @staticmethod
    def backward(ctx, grad):
        raise NotImplementedError("newton_schulz has no gradient: detach its input")


def embedding_lookup_workspace_bytes(T: int) -> int:
    return int(_load().tgs_embedding_lookup_workspace_bytes(T))


def embedding_lookup(tokens: torch.Tensor, table: torch.Tensor, scale: float = 1.0, out_dtype=None, out=None,
                     ws: torch.Tensor | None = None) -> torch.Tensor:
    """Rows of an embedding table: ``out[..., :] = scale * table[tokens[...]]``.

    ``tokens`` (int32 or int64, any shape) index ``table`` (fp32, bf16 or
    fp16, ``[V, D]``); a negative token is a masked place and gives a row of
    zeros.  ``out`` has the shape ``tokens.shape + (D,)`` and the type
    ``out_dtype`` (the table's if not given).  A token >= V gives zeros and
    sets the bad-input bit that ``check_device_error(ws)`` reports.

    Differentiable in the table, whose gradient is ``embedding_grad``'s, in the
    table's type; not with ``out``."""
    _require_any(table, _FLOATS, "table")
    dev = table.device
    _require_any(tokens, _TOKENS, "tokens", dev)
    if table.dim() != 2:
        raise ValueError("table must have shape [V, D]")
    V, D = table.shape
    if table.requires_grad and _differentiable("table", out):
        return _Lookup.apply(tokens, table, scale, out_dtype, ws)
    given = out is not None
    if not given:
        out_dtype = out_dtype or table.dtype
        if out_dtype not in _FLOATS:
            raise TypeError("out_dtype must be one of %s" % ", ".join(map(str, _FLOATS)))
        out = table.new_empty((*tokens.shape, D), dtype=out_dtype)
    else:
        _require_any(out, _FLOATS if out_dtype is None else (out_dtype,), "out", dev)
        if out.shape != (*tokens.shape, D):
            raise ValueError("out must have shape %s" % ((*tokens.shape, D),))
    stream = _stream_handle(dev)
    if ws is None:
        ws = _scratch("embedding", 32768, dev, stream)
    else:
        _require_ws(ws, dev)
    st = _load().tgs_embedding_lookup(tokens.data_ptr(), _DTYPES[tokens.dtype], tokens.numel(), table.data_ptr(),
                                      _DTYPES[table.dtype], V, D, scale, out.data_ptr(), _DTYPES[out.dtype],
                                      ws.data_ptr(), ws.numel(), stream)
    if st:
        _check(st, "tgs_embedding_lookup")
    if given:
        _written(out)
    return out


def embedding_grad_workspace_bytes(T: int, V: int, D: int, grad_dtype=torch.float32, out_dtype=torch.float32) -> int:
    return int(_load().tgs_embedding_grad_workspace_bytes(T, V, D, _DTYPES[grad_dtype], _DTYPES[out_dtype]))


def embedding_grad(tokens: torch.Tensor, grad: torch.Tensor, num_rows: int, scale: float = 1.0, out_dtype=None,
                   out=None, accumulate: bool = False, ws: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of ``embedding_lookup`` with respect to its table:
    ``out[v] = scale * (sum of grad[t] over the places with tokens[t] == v)``,
    added to ``out`` with ``accumulate``.

    ``grad`` has the shape ``tokens.shape + (D,)``; ``out`` is
    ``[num_rows, D]`` of type ``out_dtype`` (fp32 if not given, so the result
    feeds the sparsifier's steps).  Sums are fp32 in a fixed order: equal
    inputs give equal bits.  Masked places (negative tokens) add to nothing;
    tokens >= num_rows neither, and set the bad-input bit that
    ``check_device_error(ws)`` reports.  Differentiable in ``grad``, without
    ``out``."""
    _require_any(grad, _FLOATS, "grad")
    dev = grad.device
    _require_any(tokens, _TOKENS, "tokens", dev)
    if grad.dim() < 1 or grad.shape[:-1] != tokens.shape:
        raise ValueError("grad must have the shape of tokens and one dimension more")
    V, D = int(num_rows), grad.shape[-1]
    if grad.requires_grad and _differentiable("grad", out):
        if accumulate:
            raise ValueError("accumulate needs out")
        return _LookupGrad.apply(tokens, grad, V, scale, out_dtype, ws)
    given = out is not None
    if not given:
        if accumulate:
            raise ValueError("accumulate needs out")
        out_dtype = out_dtype or torch.float32
        if out_dtype not in _FLOATS:
            raise TypeError("out_dtype must be one of %s" % ", ".join(map(str, _FLOATS)))
        out = grad.new_empty((V, D), dtype=out_dtype)
    else:
        _require_any(out, _FLOATS if out_dtype is None else (out_dtype,), "out", dev)
        if out.shape != (V, D):
            raise ValueError("out must have shape %s" % ((V, D),))
    stream = _stream_handle(dev)
    lib = _load()
    T, gt, ot = tokens.numel(), _DTYPES[grad.dtype], _DTYPES[out.dtype]
    if ws is None:
        need = lib.tgs_embedding_grad_workspace_bytes(T, V, D, gt, ot)
        if need == 0:
            raise ValueError("invalid sizes T=%d num_rows=%d D=%d" % (T, V, D))
        ws = _scratch("embedding", need, dev, stream)
    else:
        _require_ws(ws, dev)
    st = lib.tgs_embedding_grad(tokens.data_ptr(), _DTYPES[tokens.dtype], T, grad.data_ptr(), gt, V, D, scale,
                                out.data_ptr(), ot, bool(accumulate), ws.data_ptr(), ws.numel(), stream)
    if st:
        _check(st, "tgs_embedding_grad")
    if given:
        _written(out)
    return out


NEWTON_SCHULZ_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _matrices(t, name):
    """(batch, rows, cols) of a matrix or a stack of matrices."""
    if t.dim() == 2:
        return 1, t.shape[0], t.shape[1]
    if t.dim() == 3:
        return t.shape[0], t.shape[1], t.shape[2]
    raise ValueError("%s must have shape [rows, cols] or [batch, rows, cols]" % name)


def newton_schulz_workspace_bytes(batch: int, rows: int, cols: int, dtype=torch.float32) -> int:
    return int(_load().tgs_newton_schulz_workspace_bytes(batch, rows, cols, _DTYPES[dtype]))


def newton_schulz(x: torch.Tensor, steps: int = 5, coefficients=NEWTON_SCHULZ_COEFFICIENTS, eps: float = 1e-7,
                  out=None, ws: torch.Tensor | None = None) -> torch.Tensor:
    """Orthogonalises a matrix, or each of a stack of matrices: ``X = x /
    (|x|_F + eps)``, then ``steps`` times ``X <- a X + (b A + c A^2) X`` with
    ``A = X X^T`` (over the shorter side).  ``out`` has ``x``'s shape and type
    (fp32, bf16, fp16) and may be ``x`` itself.  Going back through it raises:
    it has no gradient."""
    _require_any(x, _FLOATS, "x")
    dev = x.device
    b, m, n = _matrices(x, "x")
    if x.requires_grad and _differentiable("x", out):
        return _NewtonSchulz.apply(x, steps, coefficients, eps, ws)
    given = out is not None
    if not given:
        out = torch.empty_like(x)
    else:
        _require_any(out, (x.dtype,), "out", dev)
        if out.shape != x.shape:
            raise ValueError("out must have x's shape")
    if x.numel() == 0:
        return out
    stream = _stream_handle(dev)
    lib = _load()
    dt = _DTYPES[x.dtype]
    if ws is None:
        need = lib.tgs_newton_schulz_workspace_bytes(b, m, n, dt)
        if need == 0:
            raise ValueError("invalid sizes batch=%d rows=%d cols=%d" % (b, m, n))
        ws = _scratch("muon", need, dev, stream)
    else:
        _require_ws(ws, dev)
    ca, cb, cc = coefficients
    st = lib.tgs_newton_schulz(x.data_ptr(), dt, b, m, n, steps, ca, cb, cc, eps, out.data_ptr(), ws.data_ptr(),
                               ws.numel(), stream)
    if st:
        _check(st, "tgs_newton_schulz")
    if given:
        _written(out)
    return out


def muon_workspace_bytes(batch: int, rows: int, cols: int, weight_dtype=torch.float32) -> int:
    return int(_load().tgs_muon_workspace_bytes(batch, rows, cols, _DTYPES[weight_dtype]))


def muon_step(weight: torch.Tensor, grad: torch.Tensor, momentum: torch.Tensor, lr: float, beta: float = 0.95,
              nesterov: bool = True, weight_decay: float = 0.0, steps: int = 5,
              coefficients=NEWTON_SCHULZ_COEFFICIENTS, eps: float = 1e-7, ws: torch.Tensor | None = None):
    """One Muon step for a weight matrix, or a stack of them: ``momentum <-
    beta momentum + grad``, ``u = grad + beta momentum`` (or ``momentum``
    without ``nesterov``), ``O = newton_schulz(u)``, ``weight <- (1 - lr
    weight_decay) weight - lr sqrt(max(1, rows / cols)) O``.  ``weight`` and
    ``grad`` are fp32, bf16 or fp16, ``momentum`` is fp32; weight and momentum
    are updated in place.  Rows are taken to be a layer's outputs: for a matrix
    kept as ``[in, out]`` the factor is the caller's, through ``lr``.  Returns
    ``weight``."""
    _require_any(weight, _FLOATS, "weight")
    dev = weight.device
    _require_any(grad, _FLOATS, "grad", dev)
    _require_any(momentum, (torch.float32,), "momentum", dev)
    b, m, n = _matrices(weight, "weight")
    if grad.shape != weight.shape or momentum.shape != weight.shape:
        raise ValueError("weight, grad and momentum must have one shape")
    if weight.numel() == 0:
        return weight
    stream = _stream_handle(dev)
    lib = _load()
    wt = _DTYPES[weight.dtype]
    if ws is None:
        need = lib.tgs_muon_workspace_bytes(b, m, n, wt)
        if need == 0:
            raise ValueError("invalid sizes batch=%d rows=%d cols=%d" % (b, m, n))
        ws = _scratch("muon", need, dev, stream)
    else:
        _require_ws(ws, dev)
    ca, cb, cc = coefficients
    st = lib.tgs_muon_step(weight.data_ptr(), wt, grad.data_ptr(), _DTYPES[grad.dtype], momentum.data_ptr(), b, m, n,
                           lr, beta, bool(nesterov), weight_decay, steps, ca, cb, cc, eps, ws.data_ptr(), ws.numel(),
                           stream)
    if st:
        _check(st, "tgs_muon_step")
    _written(weight)
    _written(momentum)
    return weight


# ------------------------------------------ rows, from hidden states to losses --
def _call(dev, entry, *args):
    """A C entry's status; launches go to the current device, which is the tensors' own for the time of the call."""
    if dev.index == torch._C._cuda_getDevice():
        return entry(*args)
    with torch.cuda.device(dev):
        return entry(*args)


class _NoWayBack(torch.autograd.Function):
    """The result of a call that has no gradient, on inputs that require one: going back through it raises."""

    @staticmethod
    def forward(ctx, what, call, *inputs):
        ctx.what = what
        return call()

    @staticmethod
    def backward(ctx, *grads):
        raise NotImplementedError("%s has no gradient: detach its inputs" % ctx.what)


def _tracked(*tensors) -> bool:
    if torch.is_grad_enabled():
        for t in tensors:
            if t is not None and t.requires_grad:
                return True
    return False


def _untracked_out(out):
    """A graph that ``out`` belongs to would go back through values that are no longer there."""
    if _tracked(out):
        raise RuntimeError("out requires a gradient, which a call with out= has not")


@functools.lru_cache(maxsize=1024)
def _need(query, *sizes) -> int:
    """What a workspace query of the library says of these sizes and types."""
    return int(getattr(_load(), query)(*sizes))


def _spaced_rows(t, name, dtypes, device=None):
    """(rows, columns, elements from row to row) of ``[..., V]``, whose rows may lie further apart than they are long."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if forward_ad._current_level >= 0:  # a level of forward mode is open
        _no_tangent(t, name)
    if t.dtype not in dtypes:
        raise TypeError("%s must be one of %s, got %s" % (name, ", ".join(map(str, dtypes)), t.dtype))
    if not t.is_cuda:
        raise TypeError("%s must be a GPU tensor" % name)
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    if t.dim() < 1:
        raise ValueError("%s must have a last axis of scores" % name)
    V = t.shape[-1]
    rows = t.numel() // V if V else 0
    if t.is_contiguous():
        return rows, V, V
    if V > 1 and t.stride(-1) != 1:
        raise ValueError("%s must be contiguous along its last axis" % name)
    gap = run = None  # elements from row to row; from one index of the next axis to another
    for size, stride in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if size == 1:
            continue
        if gap is None:
            gap = run = stride
        if stride != run:
            raise ValueError("%s must have rows a fixed number of elements apart" % name)
        run = stride * size
    gap = V if gap is None else gap
    if gap < V:
        raise ValueError("%s has rows that overlap" % name)
    return rows, V, gap


def _places(t, dtypes, name, device, shape):
    _require_any(t, dtypes, name, device)
    if t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))


def _rows_out(logits, out):
    """(out, its elements from row to row, whether it was given) of a gradient of ``logits``."""
    if out is None:
        return logits.new_empty(logits.shape), logits.shape[-1], False
    _, _, gap = _spaced_rows(out, "out", (logits.dtype,), logits.device)
    if out.shape != logits.shape:
        raise ValueError("out must have shape %s" % (tuple(logits.shape),))
    _untracked_out(out)
    return out, gap, True


def _row_scratch(ws, need, dev, stream, what):
    if need == 0:
        raise ValueError("invalid sizes of %s" % what)
    if ws is None:
        return _scratch("rows", need, dev, stream)
    _require_ws(ws, dev)
    return ws


class _LayerNorm(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, weight, bias, eps, out_dtype):
        y, mean, rstd = layer_norm(x, weight, bias, eps, out_dtype, return_stats=True)
        ctx.save_for_backward(x, weight, mean, rstd)
        ctx.param_dtype = (weight if weight is not None else bias).dtype if (
            weight is not None or bias is not None) else None
        ctx.mark_non_differentiable(mean, rstd)
        ctx.set_materialize_grads(False)
        return y, mean, rstd

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, _mean, _rstd):
        if grad is None:
            return None, None, None, None, None
        x, weight, mean, rstd = ctx.saved_tensors
        _, need_w, need_b = ctx.needs_input_grad[:3]
        gx, gw, gb = layer_norm_grad(grad.contiguous(), x, mean, rstd, weight, params=need_w or need_b,
                                     param_dtype=ctx.param_dtype)
        return gx, gw if need_w else None, gb if need_b else None, None, None


def layer_norm(x: torch.Tensor, weight: torch.Tensor | None = None, bias: torch.Tensor | None = None,
               eps: float = 1e-5, out_dtype=None, out=None, return_stats: bool = False):
    """Layer norm over the last axis: ``(x - mean) * rstd * weight + bias``
    with ``rstd = 1 / sqrt(var + eps)``.

    ``x`` is fp32, bf16 or fp16; ``weight`` and ``bias`` (``[D]``, one type of
    the three) may each be left out.  The result has ``x``'s shape and the type
    ``out_dtype`` (``x``'s if not given); ``out`` may be ``x`` itself.  With
    ``return_stats`` the call returns ``(y, mean, rstd)``, fp32 of the shape
    ``x.shape[:-1]``, as ``layer_norm_grad`` takes them.  Sums are fp32.

    Differentiable in ``x``, ``weight`` and ``bias``; not with ``out``."""
    _require_any(x, _FLOATS, "x")
    dev = x.device
    if x.dim() < 1:
        raise ValueError("x must have a last axis")
    D = x.shape[-1]
    wt = None
    for p, name in ((weight, "weight"), (bias, "bias")):
        if p is None:
            continue
        _places(p, _FLOATS if wt is None else (wt,), name, dev, (D,))
        wt = p.dtype
    if _tracked(x, weight, bias):
        if out is not None:
            raise RuntimeError("an input requires a gradient, which a call with out= has not")
        y, mean, rstd = _LayerNorm.apply(x, weight, bias, eps, out_dtype)
        return (y, mean, rstd) if return_stats else y
    given = out is not None
    if not given:
        out_dtype = out_dtype or x.dtype
        if out_dtype not in _FLOATS:
            raise TypeError("out_dtype must be one of %s" % ", ".join(map(str, _FLOATS)))
        out = torch.empty_like(x, dtype=out_dtype)
    else:
        _places(out, _FLOATS if out_dtype is None else (out_dtype,), "out", dev, x.shape)
        _untracked_out(out)
    mean = rstd = None
    if return_stats:
        mean, rstd = x.new_empty((2, *x.shape[:-1]), dtype=torch.float32).unbind()
    st = _call(dev, _load().tgs_layer_norm, x.data_ptr(), _DTYPES[x.dtype], x.numel() // D if D else 0, D,
               None if weight is None else weight.data_ptr(), None if bias is None else bias.data_ptr(),
               0 if wt is None else _DTYPES[wt], eps, out.data_ptr(), _DTYPES[out.dtype], _ptr(mean), _ptr(rstd),
               _stream_handle(dev))
    if st:
        _check(st, "tgs_layer_norm")
    if given:
        _written(out)
    return (out, mean, rstd) if return_stats else out


def layer_norm_grad_workspace_bytes(T: int, D: int) -> int:
    return int(_load().tgs_layer_norm_grad_workspace_bytes(T, D))


def layer_norm_grad(grad: torch.Tensor, x: torch.Tensor, mean: torch.Tensor, rstd: torch.Tensor,
                    weight: torch.Tensor | None = None, params: bool = True, param_dtype=None, out=None,
                    ws: torch.Tensor | None = None):
    """The gradients of ``layer_norm``: ``(grad_x, grad_weight, grad_bias)``.

    ``grad`` has ``x``'s shape, ``mean`` and ``rstd`` are what the forward pass
    left.  ``grad_x`` has ``x``'s type and may go to ``out``, which may be ``x``
    or (of the same type) ``grad`` itself.  ``grad_weight`` and ``grad_bias``
    are sums over all rows, ``[D]`` of ``param_dtype`` (``weight``'s type, fp32
    without one), and ``None`` unless ``params``.  Sums are fp32 in a fixed
    order: equal inputs give equal bits.  It has no gradient itself."""
    _require_any(x, _FLOATS, "x")
    dev = x.device
    if x.dim() < 1:
        raise ValueError("x must have a last axis")
    D = x.shape[-1]
    _places(grad, _FLOATS, "grad", dev, x.shape)
    _places(mean, (torch.float32,), "mean", dev, x.shape[:-1])
    _places(rstd, (torch.float32,), "rstd", dev, x.shape[:-1])
    if weight is not None:
        _places(weight, _FLOATS, "weight", dev, (D,))
    if _tracked(grad, x, mean, rstd, weight):
        if out is not None:
            raise RuntimeError("an input requires a gradient, which a call with out= has not")
        results = _NoWayBack.apply("layer_norm_grad", lambda: tuple(
            r for r in layer_norm_grad(grad, x, mean, rstd, weight, params, param_dtype, ws=ws) if r is not None),
            grad, x, mean, rstd, weight)
        return results if params else (results[0], None, None)
    given = out is not None
    if not given:
        out = torch.empty_like(x)
    else:
        _places(out, (x.dtype,), "out", dev, x.shape)
        _untracked_out(out)
    gw = gb = None
    if params:
        param_dtype = param_dtype or (torch.float32 if weight is None else weight.dtype)
        if param_dtype not in _FLOATS:
            raise TypeError("param_dtype must be one of %s" % ", ".join(map(str, _FLOATS)))
        gw, gb = x.new_empty(D, dtype=param_dtype), x.new_empty(D, dtype=param_dtype)
    T = x.numel() // D if D else 0
    stream = _stream_handle(dev)
    ws = _row_scratch(ws, _need("tgs_layer_norm_grad_workspace_bytes", T, D), dev, stream, "layer_norm_grad")
    st = _call(dev, _load().tgs_layer_norm_grad, grad.data_ptr(), _DTYPES[grad.dtype], x.data_ptr(), _DTYPES[x.dtype],
               T, D, mean.data_ptr(), rstd.data_ptr(), None if weight is None else weight.data_ptr(),
               0 if weight is None else _DTYPES[weight.dtype], out.data_ptr(), _ptr(gw), _ptr(gb),
               _DTYPES[param_dtype] if params else 0, ws.data_ptr(), ws.numel(), stream)
    if st:
        _check(st, "tgs_layer_norm_grad")
    if given:
        _written(out)
    return out, gw, gb


class TokenLogprobs(NamedTuple):
    """What ``token_logprobs`` returns; what was not asked for is ``None``."""
    logprobs: torch.Tensor
    entropy: torch.Tensor | None
    top_logprobs: torch.Tensor | None
    top_indices: torch.Tensor | None
    stats: torch.Tensor


class _TokenLogprobs(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, tokens, temperature, top, entropy, ws):
        r = token_logprobs(logits, tokens, temperature, top, entropy, ws)
        ctx.save_for_backward(logits, tokens, r.stats, r.entropy)
        ctx.temperature = temperature
        ctx.mark_non_differentiable(*(t for t in (r.top_logprobs, r.top_indices, r.stats) if t is not None))
        ctx.set_materialize_grads(False)
        return tuple(r)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, grad_entropy, *_):
        if grad is None and grad_entropy is None:
            return None, None, None, None, None, None
        logits, tokens, stats, entropy = ctx.saved_tensors
        grads = (None if g is None else g.contiguous() for g in (grad, grad_entropy))
        g, ge = grads
        return token_logprobs_grad(logits, tokens, stats, g, entropy, ge, ctx.temperature), None, None, None, None, None


def token_logprobs_workspace_bytes(T: int, V: int, dtype=torch.float32, top: int = 0) -> int:
    return int(_load().tgs_token_logprobs_workspace_bytes(T, V, _DTYPES[dtype], top))


def token_logprobs(logits: torch.Tensor, tokens: torch.Tensor, temperature: float = 1.0, top: int = 0,
                   entropy: bool = False, ws: torch.Tensor | None = None) -> TokenLogprobs:
    """Log probabilities of given tokens under ``softmax(logits / temperature)``.

    ``logits`` (fp32, bf16 or fp16, ``[..., V]``) may be a view whose rows lie
    further apart than they are long (a padded vocabulary); ``tokens`` (int32 or
    int64) has the shape ``logits.shape[:-1]``.  Returns a ``TokenLogprobs``
    of fp32 ``logprobs``, with ``entropy`` the distribution's entropy, with
    ``top`` (up to 64) the rows' largest scores as ``top_indices`` (int32, ties
    to the lower index) and ``top_logprobs``, ``[..., top]``; and ``stats``, as
    ``token_logprobs_grad`` takes them.

    A negative token is a masked place: its row is not needed and its results are
    0 (alternatives -1); a token >= V too, and it sets the bad-input bit that
    ``check_device_error(ws)`` reports.  Scores of -inf have no probability.

    Differentiable in ``logits`` through ``logprobs`` and ``entropy``."""
    T, V, gap = _spaced_rows(logits, "logits", _FLOATS)
    dev = logits.device
    _places(tokens, _TOKENS, "tokens", dev, logits.shape[:-1])
    if _tracked(logits):
        return TokenLogprobs(*_TokenLogprobs.apply(logits, tokens, temperature, top, entropy, ws))
    top = int(top)
    shape = tokens.shape
    logprobs = torch.empty_like(tokens, dtype=torch.float32)
    stats = logits.new_empty((*shape, 2), dtype=torch.float32)
    ent = torch.empty_like(logprobs) if entropy else None
    at = values = None
    if top > 0:
        at = logits.new_empty((*shape, top), dtype=torch.int32)
        values = logits.new_empty((*shape, top), dtype=torch.float32)
    dt = _DTYPES[logits.dtype]
    stream = _stream_handle(dev)
    need = _need("tgs_token_logprobs_workspace_bytes", T, V, dt, top)
    ws = _row_scratch(ws, need, dev, stream, "token_logprobs: V=%d, top=%d" % (V, top) if need == 0 else "")
    st = _call(dev, _load().tgs_token_logprobs, logits.data_ptr(), dt, T, V, gap, tokens.data_ptr(),
               _DTYPES[tokens.dtype], temperature, logprobs.data_ptr(), stats.data_ptr(), _ptr(ent), top, _ptr(at),
               _ptr(values), ws.data_ptr(), ws.numel(), stream)
    if st:
        _check(st, "tgs_token_logprobs")
    return TokenLogprobs(logprobs, ent, values, at, stats)


def token_logprobs_grad(logits: torch.Tensor, tokens: torch.Tensor, stats: torch.Tensor,
                        grad_logprobs: torch.Tensor | None = None, entropy: torch.Tensor | None = None,
                        grad_entropy: torch.Tensor | None = None, temperature: float = 1.0, out=None,
                        ws: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of ``token_logprobs`` with respect to its logits:
    ``(grad_logprobs (onehot(token) - p) - grad_entropy p (log p + entropy)) /
    temperature``, of the logits' type and shape.

    ``stats`` (and ``entropy``, with ``grad_entropy``) are what the forward pass
    left; either incoming gradient may be left out.  ``out`` may be the logits
    themselves, which are then overwritten.  Masked places, and rows of which
    every score is -inf, give zeros; NaN or +inf in another row makes its gradient
    NaN.  It has no gradient itself."""
    T, V, gap = _spaced_rows(logits, "logits", _FLOATS)
    dev = logits.device
    shape = logits.shape[:-1]
    _places(tokens, _TOKENS, "tokens", dev, shape)
    _places(stats, (torch.float32,), "stats", dev, (*shape, 2))
    if grad_logprobs is None and grad_entropy is None:
        raise ValueError("grad_logprobs or grad_entropy must be given")
    if grad_entropy is not None and entropy is None:
        raise ValueError("grad_entropy needs entropy")
    for t, name in ((grad_logprobs, "grad_logprobs"), (entropy, "entropy"), (grad_entropy, "grad_entropy")):
        if t is not None:
            _places(t, (torch.float32,), name, dev, shape)
    if _tracked(logits, stats, grad_logprobs, entropy, grad_entropy):
        if out is not None:
            raise RuntimeError("an input requires a gradient, which a call with out= has not")
        return _NoWayBack.apply("token_logprobs_grad", lambda: token_logprobs_grad(
            logits, tokens, stats, grad_logprobs, entropy, grad_entropy, temperature, ws=ws),
            logits, stats, grad_logprobs, entropy, grad_entropy)
    out, gap_out, given = _rows_out(logits, out)
    stream = _stream_handle(dev)
    ws = _row_scratch(ws, _HEADER_BYTES, dev, stream, "")
    st = _call(dev, _load().tgs_token_logprobs_grad, logits.data_ptr(), _DTYPES[logits.dtype], T, V, gap,
               tokens.data_ptr(), _DTYPES[tokens.dtype], temperature, stats.data_ptr(), _ptr(grad_logprobs),
               _ptr(entropy), _ptr(grad_entropy), out.data_ptr(), gap_out, ws.data_ptr(), ws.numel(), stream)
    if st:
        _check(st, "tgs_token_logprobs_grad")
    if given:
        _written(out)
    return out


def _slots(logits, indices, teacher):
    """(rows, V, elements from row to row, K) of a distillation's inputs."""
    T, V, gap = _spaced_rows(logits, "logits", _FLOATS)
    dev = logits.device
    _require_any(indices, _TOKENS, "teacher_indices", dev)
    if indices.dim() != logits.dim() or indices.shape[:-1] != logits.shape[:-1]:
        raise ValueError("teacher_indices must have the logits' shape but for its last axis, the slots")
    _places(teacher, _FLOATS, "teacher_logits", dev, indices.shape)
    if teacher.requires_grad and torch.is_grad_enabled():
        raise RuntimeError("the teacher has no gradient: detach teacher_logits")
    return T, V, gap, indices.shape[-1]


class _DistillationLoss(torch.autograd.Function):
    @staticmethod
    def forward(ctx, logits, indices, teacher, temperature, ws):
        loss, stats = distillation_loss(logits, indices, teacher, temperature, return_stats=True, ws=ws)
        ctx.save_for_backward(logits, indices, teacher, stats)
        ctx.temperature = temperature
        ctx.mark_non_differentiable(stats)
        ctx.set_materialize_grads(False)
        return loss, stats

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad, _stats):
        if grad is None:
            return None, None, None, None, None
        logits, indices, teacher, stats = ctx.saved_tensors
        return (distillation_grad(logits, indices, teacher, stats, grad.contiguous(), ctx.temperature), None, None,
                None, None)


def distillation_workspace_bytes(T: int, V: int, dtype=torch.float32) -> int:
    return int(_load().tgs_distillation_workspace_bytes(T, V, _DTYPES[dtype]))


def distillation_loss(logits: torch.Tensor, teacher_indices: torch.Tensor, teacher_logits: torch.Tensor,
                      temperature: float = 1.0, return_stats: bool = False, ws: torch.Tensor | None = None):
    """Distillation from a teacher's top logits: of each place KL(q || p) with
    ``p = softmax(logits / temperature)`` over the vocabulary and ``q =
    softmax(teacher_logits / temperature)`` over the place's slots.

    ``logits`` is fp32, bf16 or fp16, ``[..., V]``, rows possibly further apart
    than they are long; ``teacher_indices`` (int32 or int64) and
    ``teacher_logits`` (fp32, bf16 or fp16) are ``[..., K]``, K up to 1,024.  A
    negative index is an empty slot; an index >= V too, and it sets the
    bad-input bit that ``check_device_error(ws)`` reports; an index may stand in
    several slots.  A place without any slot is masked: loss 0, gradient 0.
    Returns the losses, fp32 of the shape ``logits.shape[:-1]``; with
    ``return_stats`` also the ``stats`` that ``distillation_grad`` takes.

    Differentiable in ``logits``."""
    T, V, gap, K = _slots(logits, teacher_indices, teacher_logits)
    dev = logits.device
    if _tracked(logits):
        loss, stats = _DistillationLoss.apply(logits, teacher_indices, teacher_logits, temperature, ws)
        return (loss, stats) if return_stats else loss
    shape = logits.shape[:-1]
    loss = logits.new_empty(shape, dtype=torch.float32)
    stats = logits.new_empty((*shape, 2), dtype=torch.float32) if return_stats else None
    dt = _DTYPES[logits.dtype]
    stream = _stream_handle(dev)
    ws = _row_scratch(ws, _need("tgs_distillation_workspace_bytes", T, V, dt), dev, stream, "distillation_loss")
    st = _call(dev, _load().tgs_distillation_loss, logits.data_ptr(), dt, T, V, gap, teacher_indices.data_ptr(),
               _DTYPES[teacher_indices.dtype], teacher_logits.data_ptr(), _DTYPES[teacher_logits.dtype], K, temperature,
               loss.data_ptr(), _ptr(stats), ws.data_ptr(), ws.numel(), stream)
    if st:
        _check(st, "tgs_distillation_loss")
    return (loss, stats) if return_stats else loss


def distillation_grad(logits: torch.Tensor, teacher_indices: torch.Tensor, teacher_logits: torch.Tensor,
                      stats: torch.Tensor, grad_loss: torch.Tensor, temperature: float = 1.0, out=None,
                      ws: torch.Tensor | None = None) -> torch.Tensor:
    """The gradient of ``distillation_loss`` with respect to its logits:
    ``grad_loss (p - q) / temperature``, of the logits' type and shape.

    ``stats`` are what the forward pass left.  ``out`` may be the logits
    themselves, which are then overwritten.  Masked places, and rows of which
    every score is -inf, give zeros; NaN or +inf in another row's logits or
    teacher makes its gradient NaN.  It has no gradient itself."""
    T, V, gap, K = _slots(logits, teacher_indices, teacher_logits)
    dev = logits.device
    _places(stats, (torch.float32,), "stats", dev, (*logits.shape[:-1], 2))
    _places(grad_loss, (torch.float32,), "grad_loss", dev, logits.shape[:-1])
    if _tracked(logits, stats, grad_loss):
        if out is not None:
            raise RuntimeError("an input requires a gradient, which a call with out= has not")
        return _NoWayBack.apply("distillation_grad", lambda: distillation_grad(
            logits, teacher_indices, teacher_logits, stats, grad_loss, temperature, ws=ws), logits, stats, grad_loss)
    out, gap_out, given = _rows_out(logits, out)
    stream = _stream_handle(dev)
    ws = _row_scratch(ws, _HEADER_BYTES, dev, stream, "")
    st = _call(dev, _load().tgs_distillation_grad, logits.data_ptr(), _DTYPES[logits.dtype], T, V, gap,
               teacher_indices.data_ptr(), _DTYPES[teacher_indices.dtype], teacher_logits.data_ptr(),
               _DTYPES[teacher_logits.dtype], K, temperature, stats.data_ptr(), grad_loss.data_ptr(), out.data_ptr(),
               gap_out, ws.data_ptr(), ws.numel(), stream)
    if st:
        _check(st, "tgs_distillation_grad")
    if given:
        _written(out)
    return out


def distillation_loss_and_grad(logits: torch.Tensor, teacher_indices: torch.Tensor, teacher_logits: torch.Tensor,
                               weights: torch.Tensor | None = None, temperature: float = 1.0, out=None,
                               ws: torch.Tensor | None = None):
    """``distillation_loss`` and the gradient of ``sum(weights * loss)`` with
    respect to the logits in one call, whose second reading of a row follows the
    first and finds what LDS and the caches still hold of it:
    ``(loss, grad)``.

    ``weights`` (fp32, ``logits.shape[:-1]``) are 1 if not given: a training
    step over N places whose loss is their mean passes 1 / N.  ``out``, for the
    gradient, may be the logits themselves, which are then overwritten.  It has
    no gradient itself."""
    T, V, gap, K = _slots(logits, teacher_indices, teacher_logits)
    dev = logits.device
    if weights is not None:
        _places(weights, (torch.float32,), "weights", dev, logits.shape[:-1])
    if _tracked(logits, weights):
        if out is not None:
            raise RuntimeError("an input requires a gradient, which a call with out= has not")
        return _NoWayBack.apply("distillation_loss_and_grad", lambda: distillation_loss_and_grad(
            logits, teacher_indices, teacher_logits, weights, temperature, ws=ws), logits, weights)
    loss = logits.new_empty(logits.shape[:-1], dtype=torch.float32)
    out, gap_out, given = _rows_out(logits, out)
    dt = _DTYPES[logits.dtype]
    stream = _stream_handle(dev)
    ws = _row_scratch(ws, _need("tgs_distillation_workspace_bytes", T, V, dt), dev, stream, "distillation_loss_and_grad")
    st = _call(dev, _load().tgs_distillation_loss_and_grad, logits.data_ptr(), dt, T, V, gap,
               teacher_indices.data_ptr(), _DTYPES[teacher_indices.dtype], teacher_logits.data_ptr(),
               _DTYPES[teacher_logits.dtype], K, temperature, _ptr(weights), loss.data_ptr(), out.data_ptr(), gap_out,
               ws.data_ptr(), ws.numel(), stream)
    if st:
        _check(st, "tgs_distillation_loss_and_grad")
    if given:
        _written(out)
    return loss, out


def check_device_error(ws: torch.Tensor):
    """Waits for the current stream, then reads and clears the workspace's
    device error word: raises ValueError for bad merge input, TgsError for a
    wait timeout or inconsistent counts."""
    lib = _load()
    _check(lib.tgs_check_device_error(ws.data_ptr(), _stream_handle(ws.device)), "tgs_check_device_error")


def set_option(option: int, value: int):
    _check(_load().tgs_set_option(option, value), "tgs_set_option")


def profile_next_call(start_event, stop_event):
    """The next topk/threshold call records these torch.cuda.Events around its
    streaming pass (on its stream)."""
    lib = _load()
    for ev in (start_event, stop_event):
        if ev is not None and not ev.cuda_event:
            ev.record()  # torch creates the HIP event lazily, on its first record
    s = start_event.cuda_event if start_event is not None else None
    e = stop_event.cuda_event if stop_event is not None else None
    _check(lib.tgs_profile_next_call(s, e), "tgs_profile_next_call")


def profile_elapsed_ms(start_event, stop_event) -> float:
    """Milliseconds between two events recorded by the library."""
    ms = ctypes.c_float()
    _check(_load().tgs_profile_elapsed_ms(start_event.cuda_event, stop_event.cuda_event, ctypes.byref(ms)),
           "tgs_profile_elapsed_ms")
    return ms.value


__all__ = [
    "TopkStep", "TopkSegments", "topk_ef_step", "topk_ef_step_segmented", "threshold_ef_step", "gtopk_merge",
    "topk_workspace_bytes", "topk_segmented_workspace_bytes", "threshold_workspace_bytes",
    "gtopk_workspace_bytes", "check_device_error", "error_word", "workspace_init", "set_option",
    "threshold_estimate", "threshold_estimate_workspace_bytes", "threshold_ef_step_dev",
    "estimated_threshold_ef_step", "rtopk_ef_step", "rtopk_workspace_bytes",
    "newton_schulz", "newton_schulz_workspace_bytes", "muon_step", "muon_workspace_bytes",
    "NEWTON_SCHULZ_COEFFICIENTS",
    "embedding_lookup", "embedding_lookup_workspace_bytes", "embedding_grad", "embedding_grad_workspace_bytes",
    "layer_norm", "layer_norm_grad", "layer_norm_grad_workspace_bytes",
    "TokenLogprobs", "token_logprobs", "token_logprobs_workspace_bytes", "token_logprobs_grad",
    "distillation_loss", "distillation_grad", "distillation_loss_and_grad", "distillation_workspace_bytes",
    "profile_next_call", "profile_elapsed_ms", "library", "workspace",
    "TgsError", "OPT_TOPK_PATH", "OPT_MAIN_GRID", "LIB_PATH",
]
