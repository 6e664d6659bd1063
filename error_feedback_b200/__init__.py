"""B200 Top-k sparsifier with error feedback and gTop-k merge.

Thin ctypes binding over the C ABI in ``include/topk_ef.h``
(``libtopk_ef.so``, built in-tree by ``python -m error_feedback_b200.build``).
The binding only marshals arguments: every step of the computation runs in
the library's CUDA kernels.  PyTorch supplies device memory and the current
stream.  There is no CPU fallback: if the library is missing or the tensors
are not on a CUDA device the calls raise.

Functions mirror the C names:

* ``topk_ef_compress(grad, residual, lr, k)``            -> (idx, val)
* ``topk_ef_compress_batched(grad, residual, offsets, k, lr)`` -> (idx, val)
* ``gtopk_merge(in_idx, in_val, k, n)``                  -> (idx, val, count)
* ``embedding_lookup(weight, ids, scale)``               -> out
* ``embedding_grad(grad_out, ids, num_rows, scale)``     -> grad_weight
* ``muon_update(grad, momentum, mu)``                    -> out
* ``embedding_grad_rows(grad_out, ids, num_rows, scale)`` -> (rows, val, count)
* ``layer_norm(x, weight, bias)``                        -> (out, mean, rstd)
* ``layer_norm_grad(grad_out, x, mean, rstd, weight)``   -> (grad_x, grad_weight, grad_bias)
* ``token_logprobs(logits, ids, scale, top)``            -> (logprob, entropy, lse, top_ids, top_logprobs)
* ``token_logprobs_grad(logits, ids, lse, ...)``         -> grad_logits
* ``distill_loss(logits, teacher_ids, teacher_logits)``  -> (loss, grad_logits)
* ``topk_ef_workspace_bytes``, ``topk_ef_batched_workspace_bytes``,
  ``gtopk_merge_workspace_bytes``, ``topk_ef_last_device_status``,
  ``topk_ef_path_info``, ``topk_ef_set_test_flags``.
"""
from __future__ import annotations

import ctypes
import os

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libtopk_ef.so")

OK = 0
ERR_INVALID_ARG = -1
ERR_WORKSPACE = -2
ERR_CUDA = -3
ERR_DEVICE_TIMEOUT = -4
ERR_BAD_INPUT = -5
ERR_INTERNAL = -6


class TopkEfError(RuntimeError):
    def __init__(self, code: int, what: str):
        self.code = code
        super().__init__(f"{what}: {status_string(code)} ({code})")


_lib = None

_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_i32 = ctypes.c_int32
_sz = ctypes.c_size_t
_pi64 = ctypes.POINTER(ctypes.c_int64)


def lib() -> ctypes.CDLL:
    """The loaded C-ABI library (raises if it has not been built)."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise ImportError(f"{LIB_PATH} is missing: run `python -m error_feedback_b200.build`")
        L = ctypes.CDLL(LIB_PATH)
        L.topk_ef_workspace_bytes.argtypes = [_i64, _i64]
        L.topk_ef_workspace_bytes.restype = _sz
        L.topk_ef_compress.argtypes = [_vp, _vp, _i64, ctypes.c_float, _i64, _vp, _vp, _vp, _sz, _vp]
        L.topk_ef_compress.restype = ctypes.c_int
        L.topk_ef_compress_static.argtypes = [_vp, _vp, _i64, ctypes.c_float, _i64, _vp, _vp,
                                              _vp]
        L.topk_ef_compress_static.restype = ctypes.c_int
        L.topk_ef_static_last_device_status.argtypes = [_vp]
        L.topk_ef_static_last_device_status.restype = ctypes.c_int
        L.topk_ef_threshold_workspace_bytes.argtypes = [_i64]
        L.topk_ef_threshold_workspace_bytes.restype = _sz
        L.topk_ef_threshold.argtypes = [_vp, _vp, _i64, ctypes.c_float, ctypes.c_float, _i64,
                                        _vp, _vp, _vp, _vp, _sz, _vp]
        L.topk_ef_threshold.restype = ctypes.c_int
        L.gtopk_residual_return_workspace_bytes.argtypes = []
        L.gtopk_residual_return_workspace_bytes.restype = _sz
        L.gtopk_residual_return.argtypes = [_vp, _vp, _i32, _i64, _vp, _i64, _vp, _i64, _vp,
                                            _sz, _vp]
        L.gtopk_residual_return.restype = ctypes.c_int
        L.topk_allgather_workspace_bytes.argtypes = [_i32, _i64, _i64]
        L.topk_allgather_workspace_bytes.restype = _sz
        L.topk_allgather_sum.argtypes = [_vp, _vp, _i32, _i64, _i64, _vp, _vp, _sz, _vp]
        L.topk_allgather_sum.restype = ctypes.c_int
        L.topk_ef_batched_workspace_bytes.argtypes = [_pi64, _pi64, _i32]
        L.topk_ef_batched_workspace_bytes.restype = _sz
        L.topk_ef_compress_batched.argtypes = [_vp, _vp, _pi64, _pi64, _i32, ctypes.c_float, _vp, _vp,
                                               _vp, _sz, _vp]
        L.topk_ef_compress_batched.restype = ctypes.c_int
        L.gtopk_merge_workspace_bytes.argtypes = [_i32, _i64, _i64]
        L.gtopk_merge_workspace_bytes.restype = _sz
        L.gtopk_merge.argtypes = [_vp, _vp, _i32, _i64, _i64, _i64, _vp, _vp, _vp, _vp, _sz, _vp]
        L.gtopk_merge.restype = ctypes.c_int
        L.topk_ef_last_device_status.argtypes = [_vp, _vp]
        L.topk_ef_last_device_status.restype = ctypes.c_int
        L.topk_ef_last_cuda_error.argtypes = []
        L.topk_ef_last_cuda_error.restype = ctypes.c_int
        L.topk_ef_status_string.argtypes = [ctypes.c_int]
        L.topk_ef_status_string.restype = ctypes.c_char_p
        L.topk_ef_path_info.argtypes = [_vp, _vp, _pi64]
        L.topk_ef_path_info.restype = ctypes.c_int
        L.topk_ef_phase_times.argtypes = [_vp, _vp, _pi64]
        L.topk_ef_phase_times.restype = ctypes.c_int
        L.topk_ef_set_test_flags.argtypes = [ctypes.c_int]
        L.topk_ef_set_test_flags.restype = ctypes.c_int
        L.topk_ef_trace_enable.argtypes = [ctypes.c_int]
        L.topk_ef_trace_enable.restype = ctypes.c_int
        L.topk_ef_trace_read.argtypes = [ctypes.POINTER(ctypes.c_float),
                                         ctypes.POINTER(ctypes.c_char_p), ctypes.c_int,
                                         ctypes.POINTER(ctypes.c_int)]
        L.topk_ef_trace_read.restype = ctypes.c_int
        L.topk_ef_trace_only.argtypes = [ctypes.c_char_p, ctypes.c_int]
        L.topk_ef_trace_only.restype = ctypes.c_int
        L.embedding_lookup_workspace_bytes.argtypes = []
        L.embedding_lookup_workspace_bytes.restype = _sz
        L.embedding_lookup.argtypes = [_vp, _i32, _i64, _vp, _i32, _i64, _i64, _i64,
                                       ctypes.c_float, _vp, _i32, _i64, _vp, _sz, _vp]
        L.embedding_lookup.restype = ctypes.c_int
        L.embedding_grad_workspace_bytes.argtypes = [_i64, _i64, _i64]
        L.embedding_grad_workspace_bytes.restype = _sz
        L.embedding_grad.argtypes = [_vp, _i32, _i64, _vp, _i32, _i64, _i64, _i64, ctypes.c_float,
                                     _i64, _vp, _i32, _i64, _i32, _vp, _sz, _vp]
        L.embedding_grad.restype = ctypes.c_int
        L.embedding_grad_rows.argtypes = [_vp, _i32, _i64, _vp, _i32, _i64, _i64, _i64,
                                          ctypes.c_float, _i64, _vp, _vp, _i32, _i64, _vp, _vp,
                                          _sz, _vp]
        L.embedding_grad_rows.restype = ctypes.c_int
        L.muon_workspace_bytes.argtypes = [_i32, _i64, _i64, _i32]
        L.muon_workspace_bytes.restype = _sz
        L.muon_update.argtypes = [_vp, _i32, _i64, _i64, _vp, _i32, _i64, _i64, ctypes.c_float,
                                  _i32, ctypes.c_float, ctypes.POINTER(ctypes.c_float), _i32,
                                  ctypes.c_float, _vp, _i32, _i64, _i64, _vp, _sz, _vp]
        L.muon_update.restype = ctypes.c_int
        L.layer_norm.argtypes = [_vp, _i32, _i64, _vp, _i32, _vp, _i32, _i64, _i64, ctypes.c_float,
                                 _vp, _i32, _i64, _vp, _vp, _vp]
        L.layer_norm.restype = ctypes.c_int
        L.layer_norm_grad_workspace_bytes.argtypes = [_i64, _i64]
        L.layer_norm_grad_workspace_bytes.restype = _sz
        L.layer_norm_grad.argtypes = [_vp, _i32, _i64, _vp, _i32, _i64, _vp, _vp, _vp, _i32, _i64,
                                      _i64, _vp, _i64, _vp, _i32, _vp, _i32, _i32, _vp, _sz, _vp]
        L.layer_norm_grad.restype = ctypes.c_int
        L.token_logprobs_workspace_bytes.argtypes = []
        L.token_logprobs_workspace_bytes.restype = _sz
        L.token_logprobs.argtypes = [_vp, _i32, _i64, _vp, _i32, _i64, _i64, ctypes.c_float, _i64,
                                     _i32, _vp, _vp, _vp, _vp, _vp, _vp, _sz, _vp]
        L.token_logprobs.restype = ctypes.c_int
        L.token_logprobs_grad.argtypes = [_vp, _i32, _i64, _vp, _i32, _i64, _i64, ctypes.c_float,
                                          _i64, _vp, _vp, _vp, _vp, _vp, _i32, _i64, _vp, _sz, _vp]
        L.token_logprobs_grad.restype = ctypes.c_int
        L.distill_loss_workspace_bytes.argtypes = []
        L.distill_loss_workspace_bytes.restype = _sz
        L.distill_loss.argtypes = [_vp, _i32, _i64, _vp, _i32, _vp, _i32, _i64, _i64, _i32,
                                   ctypes.c_float, _vp, _vp, _vp, _i32, _i64, _vp, _sz, _vp]
        L.distill_loss.restype = ctypes.c_int
        _lib = L
    return _lib


def status_string(code: int) -> str:
    return lib().topk_ef_status_string(int(code)).decode()


def _check(rc: int, what: str) -> None:
    if rc != OK:
        if rc == ERR_CUDA:
            raise TopkEfError(rc, f"{what} (cudaError {lib().topk_ef_last_cuda_error()})")
        raise TopkEfError(rc, what)


def _stream(stream) -> int:
    s = stream if stream is not None else torch.cuda.current_stream()
    return int(s.cuda_stream)


def _cuda_f32(t: torch.Tensor, name: str) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.float32 or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous float32")


def _host_i64(a) -> ctypes.Array:
    vals = [int(x) for x in a]
    return (ctypes.c_int64 * max(1, len(vals)))(*vals)


def _workspace(nbytes: int, device, ws):
    if ws is not None:
        if ws.numel() * ws.element_size() < nbytes:
            raise ValueError("workspace too small")
        if not ws.is_contiguous():
            raise ValueError("the workspace must be contiguous")
        return ws
    return torch.empty(max(int(nbytes), 256), dtype=torch.uint8, device=device)


# ------------------------------------------------------------------ compress

def topk_ef_workspace_bytes(n: int, k: int) -> int:
    return int(lib().topk_ef_workspace_bytes(int(n), int(k)))


def topk_ef_compress(grad, residual, lr, k, out_idx=None, out_val=None, ws=None, stream=None):
    """One EF step: acc = fmaf(lr, grad, residual); send the top-k of |acc|
    (ties to the lower index) in ascending index order; residual becomes acc
    with the sent slots zeroed.  Returns (idx int32[k], val float32[k])."""
    _cuda_f32(grad, "grad")
    _cuda_f32(residual, "residual")
    if grad.numel() != residual.numel():
        raise ValueError("grad and residual differ in size")
    n, k = grad.numel(), int(k)
    dev = grad.device
    if out_idx is None:
        out_idx = torch.empty(k, dtype=torch.int32, device=dev)
    if out_val is None:
        out_val = torch.empty(k, dtype=torch.float32, device=dev)
    nb = topk_ef_workspace_bytes(n, k)
    if nb == 0:
        raise TopkEfError(ERR_INVALID_ARG, "topk_ef_workspace_bytes")
    ws = _workspace(nb, dev, ws)
    rc = lib().topk_ef_compress(grad.data_ptr(), residual.data_ptr(), n, float(lr), k,
                                out_idx.data_ptr(), out_val.data_ptr(), ws.data_ptr(),
                                ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "topk_ef_compress")
    return out_idx, out_val


def topk_ef_compress_static(grad, residual, lr, k, out_idx=None, out_val=None, stream=None):
    """topk_ef_compress without a caller workspace: for callers that cannot
    allocate device memory.  Uses the library's fixed 32 MiB scratch array
    (shared by all calls; calls whose GPU work overlaps must not be issued)."""
    _cuda_f32(grad, "grad")
    _cuda_f32(residual, "residual")
    if grad.numel() != residual.numel():
        raise ValueError("grad and residual differ in size")
    n, k = grad.numel(), int(k)
    dev = grad.device
    if out_idx is None:
        out_idx = torch.empty(k, dtype=torch.int32, device=dev)
    if out_val is None:
        out_val = torch.empty(k, dtype=torch.float32, device=dev)
    rc = lib().topk_ef_compress_static(grad.data_ptr(), residual.data_ptr(), n, float(lr), k,
                                       out_idx.data_ptr(), out_val.data_ptr(), _stream(stream))
    _check(rc, "topk_ef_compress_static")
    return out_idx, out_val


def topk_ef_static_last_device_status(stream=None) -> int:
    """Device-side status of the last topk_ef_compress_static call on the
    current device (synchronises the stream)."""
    return int(lib().topk_ef_static_last_device_status(_stream(stream)))


def topk_ef_threshold_workspace_bytes(n: int) -> int:
    return int(lib().topk_ef_threshold_workspace_bytes(int(n)))


def topk_ef_threshold(grad, residual, lr, threshold, max_out, out_idx=None, out_val=None,
                      out_count=None, ws=None, stream=None):
    """Hard-threshold EF step: acc = fmaf(lr, grad, residual); the entries
    with |acc| >= |threshold| pass and the first max_out of them (ascending
    index) are sent, their residual zeroed.  Returns (idx int32[max_out],
    val float32[max_out], count int64[1] on the device); only the first
    min(count, max_out) slots of idx / val are written."""
    _cuda_f32(grad, "grad")
    _cuda_f32(residual, "residual")
    if grad.numel() != residual.numel():
        raise ValueError("grad and residual differ in size")
    n, max_out = grad.numel(), int(max_out)
    dev = grad.device
    if out_idx is None:
        out_idx = torch.empty(max(max_out, 1), dtype=torch.int32, device=dev)[:max_out]
    if out_val is None:
        out_val = torch.empty(max(max_out, 1), dtype=torch.float32, device=dev)[:max_out]
    if out_count is None:
        out_count = torch.empty(1, dtype=torch.int64, device=dev)
    nb = topk_ef_threshold_workspace_bytes(n)
    if nb == 0:
        raise TopkEfError(ERR_INVALID_ARG, "topk_ef_threshold_workspace_bytes")
    ws = _workspace(nb, dev, ws)
    rc = lib().topk_ef_threshold(grad.data_ptr(), residual.data_ptr(), n, float(lr),
                                 float(threshold), max_out, out_idx.data_ptr(),
                                 out_val.data_ptr(), out_count.data_ptr(), ws.data_ptr(),
                                 ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "topk_ef_threshold")
    return out_idx, out_val, out_count


def gtopk_residual_return_workspace_bytes() -> int:
    return int(lib().gtopk_residual_return_workspace_bytes())


def gtopk_residual_return(sent_idx, sent_val, global_idx, residual, ws=None, stream=None):
    """After gTop-k: for every worker p (row of sent_idx / sent_val) and sent
    (i, v) with i not in global_idx, residual[p, i] += v.  residual is a
    [P, n] float32 CUDA tensor, updated in place."""
    for t, name in ((sent_idx, "sent_idx"), (global_idx, "global_idx")):
        if not t.is_cuda or t.dtype != torch.int32 or not t.is_contiguous():
            raise TypeError(f"{name} must be a contiguous int32 CUDA tensor")
    _cuda_f32(sent_val, "sent_val")
    _cuda_f32(residual, "residual")
    P, k_sent = sent_idx.shape
    if residual.dim() != 2 or residual.shape[0] != P or tuple(sent_val.shape) != (P, k_sent):
        raise ValueError("shapes: sent_idx/sent_val [P, k_sent], residual [P, n]")
    n = residual.shape[1]
    ws = _workspace(gtopk_residual_return_workspace_bytes(), residual.device, ws)
    rc = lib().gtopk_residual_return(sent_idx.data_ptr(), sent_val.data_ptr(), P, k_sent,
                                     global_idx.data_ptr(), global_idx.numel(),
                                     residual.data_ptr(), n, ws.data_ptr(),
                                     ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "gtopk_residual_return")
    return ws


def topk_allgather_workspace_bytes(P: int, k_in: int, n: int) -> int:
    return int(lib().topk_allgather_workspace_bytes(int(P), int(k_in), int(n)))


def topk_allgather_sum(in_idx, in_val, n, out=None, ws=None, stream=None):
    """Dense rank-order sum of the P sets (rows of in_idx / in_val) into a
    float32[n] CUDA tensor (the AllGather aggregation)."""
    if not in_idx.is_cuda or in_idx.dtype != torch.int32 or not in_idx.is_contiguous():
        raise TypeError("in_idx must be a contiguous int32 CUDA tensor")
    _cuda_f32(in_val, "in_val")
    P, k_in = in_idx.shape
    n = int(n)
    if out is None:
        out = torch.empty(max(n, 1), dtype=torch.float32, device=in_idx.device)[:n]
    nb = topk_allgather_workspace_bytes(P, k_in, n)
    if nb == 0:
        raise TopkEfError(ERR_INVALID_ARG, "topk_allgather_workspace_bytes")
    ws = _workspace(nb, in_idx.device, ws)
    rc = lib().topk_allgather_sum(in_idx.data_ptr(), in_val.data_ptr(), P, k_in, n,
                                  out.data_ptr(), ws.data_ptr(), ws.numel() * ws.element_size(),
                                  _stream(stream))
    _check(rc, "topk_allgather_sum")
    return out


def topk_ef_batched_workspace_bytes(offsets, k) -> int:
    T = len(k)
    return int(lib().topk_ef_batched_workspace_bytes(_host_i64(offsets), _host_i64(k), T))


def topk_ef_compress_batched(grad, residual, offsets, k, lr, out_idx=None, out_val=None,
                             ws=None, stream=None):
    """Per-tensor EF step over a flat bucket (tensor l = [offsets[l],
    offsets[l+1])).  Outputs are packed in tensor order with indices local to
    each tensor.  Returns (idx int32[sum k], val float32[sum k])."""
    _cuda_f32(grad, "grad")
    _cuda_f32(residual, "residual")
    offs = _host_i64(offsets)
    ks = _host_i64(k)
    T = len(k)
    total = int(sum(int(x) for x in k))
    dev = grad.device
    if out_idx is None:
        out_idx = torch.empty(total, dtype=torch.int32, device=dev)
    if out_val is None:
        out_val = torch.empty(total, dtype=torch.float32, device=dev)
    nb = int(lib().topk_ef_batched_workspace_bytes(offs, ks, T))
    if nb == 0:
        raise TopkEfError(ERR_INVALID_ARG, "topk_ef_batched_workspace_bytes")
    ws = _workspace(nb, dev, ws)
    rc = lib().topk_ef_compress_batched(grad.data_ptr(), residual.data_ptr(), offs, ks, T,
                                        float(lr), out_idx.data_ptr(), out_val.data_ptr(),
                                        ws.data_ptr(), ws.numel() * ws.element_size(),
                                        _stream(stream))
    _check(rc, "topk_ef_compress_batched")
    return out_idx, out_val


# --------------------------------------------------------------------- merge

def gtopk_merge_workspace_bytes(P: int, k_in: int, k: int) -> int:
    return int(lib().gtopk_merge_workspace_bytes(int(P), int(k_in), int(k)))


def gtopk_merge(in_idx, in_val, k, n, out_idx=None, out_val=None, out_count=None, ws=None,
                stream=None):
    """gTop-k tournament over the P rows of in_idx (int32, each strictly
    ascending) / in_val (float32).  Returns (idx int32[k], val float32[k],
    count int32[1]); entries past count are -1 / 0."""
    if in_idx.dtype != torch.int32 or not in_idx.is_cuda or not in_idx.is_contiguous():
        raise ValueError("in_idx must be a contiguous int32 CUDA tensor")
    _cuda_f32(in_val, "in_val")
    if in_idx.dim() != 2 or in_idx.shape != in_val.shape:
        raise ValueError("in_idx and in_val must both be [P, k_in]")
    P, k_in = in_idx.shape
    k = int(k)
    dev = in_idx.device
    if out_idx is None:
        out_idx = torch.empty(max(k, 1), dtype=torch.int32, device=dev)[:k]
    if out_val is None:
        out_val = torch.empty(max(k, 1), dtype=torch.float32, device=dev)[:k]
    if out_count is None:
        out_count = torch.empty(1, dtype=torch.int32, device=dev)
    nb = gtopk_merge_workspace_bytes(P, k_in, k)
    if nb == 0:
        raise TopkEfError(ERR_INVALID_ARG, "gtopk_merge_workspace_bytes")
    ws = _workspace(nb, dev, ws)
    rc = lib().gtopk_merge(in_idx.data_ptr(), in_val.data_ptr(), P, k_in, k, int(n),
                           out_idx.data_ptr(), out_val.data_ptr(), out_count.data_ptr(),
                           ws.data_ptr(), ws.numel() * ws.element_size(), _stream(stream))
    _check(rc, "gtopk_merge")
    return out_idx, out_val, out_count


# ----------------------------------------------------------------- embedding

_TYPE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}


def _matrix(t, name: str, device=None):
    """Element type code and row stride of a CUDA matrix whose rows are
    contiguous (the rows themselves may be apart)."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    code = _TYPE.get(t.dtype)
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    if device is not None and t.get_device() != device.index:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dim() != 2:
        raise ValueError(f"{name} must have two dimensions")
    rows, cols = t.shape
    ld, step = t.stride()
    if cols > 1 and step != 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError(f"the rows of {name} overlap")
    return code, ld


def _token_ids(ids, device):
    if not isinstance(ids, torch.Tensor) or not ids.is_cuda or not ids.is_contiguous() \
            or ids.dtype not in (torch.int32, torch.int64):
        raise ValueError("ids must be a contiguous int32 or int64 CUDA tensor")
    if ids.get_device() != device.index:
        raise ValueError(f"ids is on {ids.device}, not on {device}")
    return 8 if ids.dtype == torch.int64 else 4, ids.numel()


class _On:
    """Makes a tensor's device current for a call and names the stream that
    the call and what it allocates belong to."""

    def __init__(self, device, stream):
        self.dev = device
        self.stream = stream
        self.guard = None

    def __enter__(self):
        if self.stream is not None:
            if self.stream.device != self.dev:
                raise ValueError(f"the stream is on {self.stream.device}, not on {self.dev}")
            self.guard = torch.cuda.stream(self.stream)      # its device too
        else:
            self.guard = torch.cuda.device(self.dev)
        self.guard.__enter__()
        return int((self.stream or torch.cuda.current_stream()).cuda_stream)

    def __exit__(self, *exc):
        self.guard.__exit__(*exc)


def _on(device, stream, call):
    """call(raw stream) with the device current; the usual case (its current
    stream, on the current device) at once."""
    if stream is None and device.index == torch._C._cuda_getDevice():
        return call(torch._C._cuda_getCurrentRawStream(device.index))
    with _On(device, stream) as st:
        return call(st)


def _on_device(ws, device):
    if ws is not None and ws.get_device() != device.index:
        raise ValueError(f"ws is on {ws.device}, not on {device}")
    if ws is not None and not ws.is_contiguous():
        raise ValueError("ws must be contiguous")       # (else it may hold less than its nbytes)


_LOOKUP_WS = 512                        # at least embedding_lookup_workspace_bytes()


def embedding_lookup_workspace_bytes() -> int:
    return int(lib().embedding_lookup_workspace_bytes())


def embedding_lookup(weight, ids, scale=1.0, out=None, out_dtype=None, ws=None, stream=None):
    """out[..., :] = scale * weight[ids[...], :], the product in fp32 and
    rounded once.  weight: [V, D] float32 / bfloat16 / float16 with contiguous
    rows; ids: int32 / int64 of any shape; out: [*ids.shape, D] (or [T, D]) in
    any of the types (default: the weight's).  An id outside [0, V) gives a
    row of zeros and ERR_BAD_INPUT from topk_ef_last_device_status(ws) (pass a
    ws to be able to ask).  The call works on the tensors' memory: autograd
    records nothing, and the gradient is embedding_grad's."""
    wt, ldw = _matrix(weight, "weight")
    dev = weight.device
    idb, T = _token_ids(ids, dev)
    V, D = weight.shape
    _on_device(ws, dev)

    def call(st):
        o = out
        if o is None:
            o = torch.empty((*ids.shape, D), dtype=out_dtype or weight.dtype, device=dev)
        elif out_dtype is not None and o.dtype != out_dtype:
            raise ValueError("out and out_dtype differ")
        o2 = o if o.dim() == 2 else o.view(-1, D) if o.numel() else o.new_empty((T, D))
        ot, ldo = _matrix(o2, "out", dev)
        if o2.shape != (T, D):
            raise ValueError(f"out must hold [{T}, {D}] elements")
        w = ws if ws is not None else _workspace(_LOOKUP_WS, dev, None)
        rc = lib().embedding_lookup(weight.data_ptr(), wt, ldw, ids.data_ptr(), idb, T, V, D,
                                    scale, o2.data_ptr(), ot, ldo, w.data_ptr(),
                                    w.nbytes, st)
        if rc != OK:
            _check(rc, "embedding_lookup")
        return o

    return _on(dev, stream, call)


def embedding_grad_workspace_bytes(T: int, V: int, D: int) -> int:
    return int(lib().embedding_grad_workspace_bytes(int(T), int(V), int(D)))


def _grad_args(grad_out, ids, num_rows):
    if isinstance(grad_out, torch.Tensor) and grad_out.dim() != 2 and grad_out.dim() > 0:
        D = grad_out.shape[-1]
        grad_out = grad_out.view(-1, D) if grad_out.numel() else grad_out.new_empty((ids.numel(), D))
    gt, ldg = _matrix(grad_out, "grad_out")
    dev = grad_out.device
    idb, T = _token_ids(ids, dev)
    if grad_out.shape[0] != T:
        raise ValueError("grad_out must hold one row for each id")
    return grad_out, gt, ldg, dev, idb, T, int(num_rows), grad_out.shape[1]


def _own_workspace(nbytes: int, device, what: str):
    """A workspace for one call that was given none."""
    if nbytes == 0:
        raise TopkEfError(ERR_INVALID_ARG, what)
    return _workspace(nbytes, device, None)


def embedding_grad(grad_out, ids, num_rows, scale=1.0, padding_idx=-1, accumulate=False, out=None,
                   out_dtype=None, ws=None, stream=None):
    """Gradient of embedding_lookup with respect to its weight:
    out[v] = (out[v] if accumulate else 0) + scale * sum of grad_out[t] over
    ids[t] == v, summed in fp32 in a fixed order and rounded once.  grad_out:
    [*ids.shape, D]; out: [num_rows, D] (default float32, the type that
    topk_ef_compress reads).  Positions whose id is padding_idx contribute
    nothing; other ids outside [0, num_rows) neither, and they give
    ERR_BAD_INPUT from topk_ef_last_device_status(ws)."""
    grad_out, gt, ldg, dev, idb, T, V, D = _grad_args(grad_out, ids, num_rows)
    if V < 0:
        raise ValueError("num_rows must not be negative")
    _on_device(ws, dev)

    def call(st):
        o = out
        if o is None:
            if accumulate:
                raise ValueError("accumulate needs out")
            o = torch.empty((V, D), dtype=out_dtype or torch.float32, device=dev)
        elif out_dtype is not None and o.dtype != out_dtype:
            raise ValueError("out and out_dtype differ")
        ot, ldo = _matrix(o, "out", dev)
        if o.shape != (V, D):
            raise ValueError(f"out must be [{V}, {D}]")
        # (a workspace that is given is checked by the call)
        w = ws if ws is not None else _own_workspace(
            embedding_grad_workspace_bytes(T, V, D), dev, "embedding_grad_workspace_bytes")
        rc = lib().embedding_grad(grad_out.data_ptr(), gt, ldg, ids.data_ptr(), idb, T, V, D,
                                  scale, int(padding_idx), o.data_ptr(), ot, ldo,
                                  1 if accumulate else 0, w.data_ptr(),
                                  w.nbytes, st)
        if rc != OK:
            _check(rc, "embedding_grad")
        return o

    return _on(dev, stream, call)


def embedding_grad_rows(grad_out, ids, num_rows, scale=1.0, padding_idx=-1, out_rows=None,
                        out_val=None, out_count=None, out_dtype=None, ws=None, stream=None):
    """The gradient of embedding_grad as a row-sparse set: the distinct ids in
    ascending order (padding_idx left out), the gradient row of each, and
    their number.  Returns (rows int32[m], val [m, D], count int32[1]) with
    m = min(T, num_rows); slots from the count on are not written."""
    grad_out, gt, ldg, dev, idb, T, V, D = _grad_args(grad_out, ids, num_rows)
    if V < 0:
        raise ValueError("num_rows must not be negative")
    _on_device(ws, dev)
    m = min(T, V)

    def call(st):
        rows, val, count = out_rows, out_val, out_count
        if rows is None:
            rows = torch.empty(m, dtype=torch.int32, device=dev)
        if val is None:
            val = torch.empty((m, D), dtype=out_dtype or torch.float32, device=dev)
        elif out_dtype is not None and val.dtype != out_dtype:
            raise ValueError("out_val and out_dtype differ")
        if count is None:
            count = torch.empty(1, dtype=torch.int32, device=dev)
        for t, name, least in ((rows, "out_rows", m), (count, "out_count", 1)):
            if not t.is_cuda or t.device != dev or t.dtype != torch.int32 or \
                    not t.is_contiguous() or t.numel() < least:
                raise ValueError(f"{name} must be a contiguous int32 tensor of {least} on {dev}")
        ot, ldo = _matrix(val, "out_val", dev)
        if val.shape[0] < m or val.shape[1] != D:
            raise ValueError(f"out_val must be [{m}, {D}]")
        w = ws if ws is not None else _own_workspace(
            embedding_grad_workspace_bytes(T, V, D), dev, "embedding_grad_workspace_bytes")
        rc = lib().embedding_grad_rows(grad_out.data_ptr(), gt, ldg, ids.data_ptr(), idb, T, V, D,
                                       scale, int(padding_idx), rows.data_ptr(), val.data_ptr(),
                                       ot, ldo, count.data_ptr(), w.data_ptr(),
                                       w.nbytes, st)
        if rc != OK:
            _check(rc, "embedding_grad_rows")
        return rows, val, count

    return _on(dev, stream, call)


# ---------------------------------------------------------------------- muon

MUON_COEFFICIENTS = (3.4445, -4.7750, 2.0315)


def _matrices(t, name: str, device=None):
    """(type code, row stride, matrix stride, (B, rows, cols)) of a CUDA
    tensor of one matrix or a batch of them with contiguous rows."""
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype not in _TYPE:
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, not on {device}")
    if t.dim() not in (2, 3):
        raise ValueError(f"{name} must be [rows, cols] or [B, rows, cols]")
    B = t.shape[0] if t.dim() == 3 else 1
    rows, cols = t.shape[-2:]
    if cols > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must have contiguous rows")
    ld = t.stride(-2) if rows > 1 else cols
    stride = t.stride(0) if B > 1 else rows * ld
    if t.numel() and (ld < cols or stride < (rows - 1) * ld + cols):
        raise ValueError(f"the rows of {name} overlap")
    return _TYPE[t.dtype], max(ld, cols), stride, (B, rows, cols)


def _coefficients(coefficients, steps):
    """float[3 * steps] of one (a, b, c) for every step, or one for each."""
    steps = int(steps)
    flat = list(coefficients)
    if flat and not hasattr(flat[0], "__len__"):
        flat = [flat] * steps
    if len(flat) != steps or any(len(c) != 3 for c in flat):
        raise ValueError("coefficients must be one (a, b, c), or one for each step")
    return (ctypes.c_float * max(1, 3 * steps))(*[float(x) for c in flat for x in c]), steps


def muon_workspace_bytes(B: int, rows: int, cols: int, out_dtype=torch.float32) -> int:
    return int(lib().muon_workspace_bytes(int(B), int(rows), int(cols), _TYPE[out_dtype]))


def muon_update(grad, momentum=None, mu=0.95, nesterov=True, coefficients=MUON_COEFFICIENTS,
                steps=5, eps=1e-7, scale=1.0, out=None, out_dtype=None, ws=None, stream=None):
    """Orthogonalised update of one matrix [rows, cols] or of each of a batch
    [B, rows, cols]: momentum = mu momentum + grad (in place, contiguous
    float32; None: u = grad), u = grad + mu momentum (nesterov) or momentum,
    X = u / (||u||_F + eps), `steps` times X <- a X + (b A + c A A) X with
    A = X X^T, out = scale X.  out: float32 (default) or float16, about as
    exact as plain float32 products, rounded once; or bfloat16, where the
    products read 11 bits of their operands if both sides are above 128 (2e-3
    to 4e-3 of the norm off, equal entries up to 7e-3; the rounding alone is
    1.65e-3).  out may be grad itself.  The call works on the tensors' memory:
    autograd records nothing."""
    gt, ldg, sg, (B, rows, cols) = _matrices(grad, "grad")
    dev = grad.device
    coef, steps = _coefficients(coefficients, steps)
    _on_device(ws, dev)
    mp = None
    if momentum is not None:
        _cuda_f32(momentum, "momentum")
        if momentum.shape != grad.shape or momentum.device != dev:
            raise ValueError("momentum must have grad's shape and device")
        mp = momentum.data_ptr()

    def call(st):
        o = out
        if o is None:
            o = torch.empty(grad.shape, dtype=out_dtype or torch.float32, device=dev)
        elif out_dtype is not None and o.dtype != out_dtype:
            raise ValueError("out and out_dtype differ")
        ot, ldo, so, _ = _matrices(o, "out", dev)
        if o.shape != grad.shape:
            raise ValueError("out must have grad's shape")
        w = ws if ws is not None else _own_workspace(
            lib().muon_workspace_bytes(B, rows, cols, ot), dev, "muon_workspace_bytes")
        rc = lib().muon_update(grad.data_ptr(), gt, ldg, sg, mp, B, rows, cols, mu,
                               1 if nesterov else 0, eps, coef, steps, scale, o.data_ptr(), ot,
                               ldo, so, w.data_ptr(), w.nbytes, st)
        if rc != OK:
            _check(rc, "muon_update")
        return o

    return _on(dev, stream, call)


# ---------------------------------------------------------------- layer norm

# (The checks of these calls ask a tensor for as little as they can: a short call is bound by
# what the host does, 9 us of which the GPU works 3.)

def _rows(t, name: str, D=None, index=None):
    """(2-d view, type code, row stride, device index, rows, columns) of [..., D]
    rows on a CUDA device (`index`, if given), one stride apart, whose elements
    are contiguous."""
    if not isinstance(t, torch.Tensor):
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dim() != 2:
        if t.dim() == 0:
            raise ValueError(f"{name} must have a dimension")
        n = t.shape[-1]
        try:
            t = t.view(-1, n) if t.numel() else t.new_empty((t.shape[:-1].numel(), n))
        except RuntimeError:
            raise ValueError(f"the rows of {name} must be one stride apart") from None
    at, code = t.get_device(), _TYPE.get(t.dtype)
    if at < 0:
        raise ValueError(f"{name} must be a CUDA tensor")
    if code is None:
        raise ValueError(f"{name} must be float32, bfloat16 or float16")
    if index is not None and at != index:
        raise ValueError(f"{name} is on {t.device}, not on cuda:{index}")
    rows, cols = t.shape
    ld, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name} must have contiguous rows")
    if rows <= 1:
        ld = cols
    elif ld < cols:
        raise ValueError(f"the rows of {name} overlap")
    if D is not None and cols != D:
        raise ValueError(f"{name} must have rows of {D}")
    return t, code, ld, at, rows, cols


def _vector(t, name: str, n: int, index: int):
    """Address and type code of a contiguous [n] tensor on the device; (None, 0)
    for None."""
    if t is None:
        return None, 0
    if isinstance(t, torch.Tensor) and t.get_device() == index and t.numel() == n \
            and t.is_contiguous():
        code = _TYPE.get(t.dtype)
        if code is None:
            raise ValueError(f"{name} must be float32, bfloat16 or float16")
        return t.data_ptr(), code
    raise ValueError(f"{name} must be a contiguous tensor of {n} on cuda:{index}")


def _f32(t, name: str, n: int, index: int):
    """Address of a contiguous float32 [n] tensor on the device; None for None."""
    if t is None:
        return None
    if isinstance(t, torch.Tensor) and t.dtype is torch.float32 and t.get_device() == index \
            and t.numel() == n and t.is_contiguous():
        return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous float32 tensor of {n} on cuda:{index}")


def _workspace_on(ws, index: int):
    if ws is not None and ws.get_device() != index:
        raise ValueError(f"ws is on {ws.device}, not on cuda:{index}")
    if ws is not None and not ws.is_contiguous():
        raise ValueError("ws must be contiguous")


def _at(index: int, stream, call):
    """_on of a device's index."""
    if stream is None and index == torch._C._cuda_getDevice():
        return call(torch._C._cuda_getCurrentRawStream(index))
    return _on(torch.device("cuda", index), stream, call)


def layer_norm(x, weight=None, bias=None, eps=1e-5, out=None, out_dtype=None, mean=None, rstd=None,
               stats=True, stream=None):
    """out = (x - mean) rstd weight + bias over the last dimension of x
    ([..., D] with contiguous rows one stride apart), mean and rstd = (variance + eps)^-1/2 of
    each row in fp32, the result rounded once.  Types: float32, bfloat16 or
    float16 each (out: x's by default).  out may be x.  Returns (out, mean,
    rstd), mean and rstd float32 [rows] for layer_norm_grad (None with
    stats=False and none given).  Autograd records nothing: the gradient is
    layer_norm_grad's."""
    x2, xt, ldx, at, T, D = _rows(x, "x")
    wp, wt = _vector(weight, "weight", D, at)
    bp, bt = _vector(bias, "bias", D, at)
    mp = _f32(mean, "mean", T, at)
    rp = _f32(rstd, "rstd", T, at)

    def call(st):
        o, m, r, ma, ra = out, mean, rstd, mp, rp
        if o is None:
            o = torch.empty(x.shape, dtype=out_dtype or x.dtype, device=x.device)
        elif out_dtype is not None and o.dtype != out_dtype:
            raise ValueError("out and out_dtype differ")
        o2, ot, ldo, _, rows, _ = _rows(o, "out", D, at)
        if rows != T:
            raise ValueError(f"out must hold [{T}, {D}] elements")
        if stats:
            if m is None:
                m = torch.empty(T, dtype=torch.float32, device=x.device)
                ma = m.data_ptr()
            if r is None:
                r = torch.empty(T, dtype=torch.float32, device=x.device)
                ra = r.data_ptr()
        rc = (_lib or lib()).layer_norm(x2.data_ptr(), xt, ldx, wp, wt, bp, bt, T, D, eps,
                                        o2.data_ptr(), ot, ldo, ma, ra, st)
        if rc != OK:
            _check(rc, "layer_norm")
        return o, m, r

    return _at(at, stream, call)


def layer_norm_grad_workspace_bytes(T: int, D: int) -> int:
    return int(lib().layer_norm_grad_workspace_bytes(int(T), int(D)))


def layer_norm_grad(grad_out, x, mean, rstd, weight=None, affine=True, accumulate=False,
                    grad_x=None, grad_weight=None, grad_bias=None, out_dtype=None, ws=None,
                    stream=None):
    """Gradient of layer_norm: (grad_x, grad_weight, grad_bias).  grad_out and x:
    [..., D]; mean, rstd: layer_norm's; grad_x: x's type, may be x or grad_out
    itself; grad_weight, grad_bias: [D] (out_dtype, default float32, the type
    that topk_ef_compress reads), added to what they hold with accumulate; both
    None with affine=False."""
    x2, xt, ldx, at, T, D = _rows(x, "x")
    g2, gt, ldg, _, rows, _ = _rows(grad_out, "grad_out", D, at)
    if rows != T:
        raise ValueError("grad_out must have x's rows")
    wp, wt = _vector(weight, "weight", D, at)
    if mean is None or rstd is None:
        raise ValueError("mean and rstd are needed")
    mp = _f32(mean, "mean", T, at)
    rp = _f32(rstd, "rstd", T, at)
    if affine and accumulate and (grad_weight is None or grad_bias is None):
        raise ValueError("accumulate needs grad_weight and grad_bias")
    _workspace_on(ws, at)

    def call(st):
        gx, gw, gb = grad_x, grad_weight, grad_bias
        if gx is None:
            gx = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        gx2, gxt, ldgx, _, rows, _ = _rows(gx, "grad_x", D, at)
        if rows != T or gxt != xt:
            raise ValueError("grad_x must have x's rows and type")
        w = ws
        if affine:
            if gw is None:
                gw = torch.empty(D, dtype=out_dtype or torch.float32, device=x.device)
            if gb is None:
                gb = torch.empty(D, dtype=out_dtype or torch.float32, device=x.device)
            if w is None:
                w = _own_workspace(layer_norm_grad_workspace_bytes(T, D), x.device,
                                   "layer_norm_grad_workspace_bytes")
        elif gw is not None or gb is not None:
            raise ValueError("affine=False has no grad_weight and grad_bias")
        gwp, gwt = _vector(gw, "grad_weight", D, at)
        gbp, gbt = _vector(gb, "grad_bias", D, at)
        rc = (_lib or lib()).layer_norm_grad(g2.data_ptr(), gt, ldg, x2.data_ptr(), xt, ldx, mp, rp, wp, wt,
                                   T, D, gx2.data_ptr(), ldgx, gwp, gwt, gbp, gbt,
                                   1 if accumulate else 0, None if w is None else w.data_ptr(),
                                   0 if w is None else w.nbytes, st)
        if rc != OK:
            _check(rc, "layer_norm_grad")
        return gx, gw, gb

    return _at(at, stream, call)


# ------------------------------------------------- losses over a vocabulary

_STATUS_WS = 512        # at least token_logprobs_workspace_bytes(), distill_loss_workspace_bytes()


def token_logprobs_workspace_bytes() -> int:
    return int(lib().token_logprobs_workspace_bytes())


def _id_list(ids, name: str, n: int, index: int):
    """Address of n contiguous int32 or int64 ids on the device, and their size."""
    if isinstance(ids, torch.Tensor) and ids.get_device() == index and ids.numel() == n \
            and ids.is_contiguous():
        if ids.dtype is torch.int64:
            return ids.data_ptr(), 8
        if ids.dtype is torch.int32:
            return ids.data_ptr(), 4
    raise ValueError(f"{name} must be {n} contiguous int32 or int64 values on cuda:{index}")


def _table(t, name: str, rows: int, cols: int, index: int, dtype):
    """Address of a contiguous [rows, cols] tensor on the device."""
    if isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == index and t.is_contiguous():
        s = t.shape
        if s == (rows, cols) or (s and s[-1] == cols and t.numel() == rows * cols):
            return t.data_ptr()
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of [{rows}, {cols}] on cuda:{index}")


def token_logprobs(logits, ids=None, scale=1.0, top=0, padding_idx=-1, logprob=None, entropy=None,
                   lse=None, top_ids=None, top_logprobs=None, ws=None, stream=None):
    """Of each row of logits ([..., V], contiguous rows one stride apart), with
    p = softmax(scale logits): (log p[ids], the entropy, the log of the sum, the ids
    of the `top` largest logits in descending order, the lower first among
    equal ones, and their log-probabilities).  The outputs are float32 [rows]
    and int32 / float32 [rows, top]; the first is None without ids, the last two
    with top=0.  Rows whose id is padding_idx are not read: 0, and ids of -1 at
    -inf.  Another id outside [0, V) gives 0 and ERR_BAD_INPUT from
    topk_ef_last_device_status(ws).  Autograd records nothing: the gradient is
    token_logprobs_grad's."""
    z, zt, ldz, at, T, V = _rows(logits, "logits")
    ip, idb = (None, 8) if ids is None else _id_list(ids, "ids", T, at)
    top = int(top)
    if ids is None and logprob is not None:
        raise ValueError("logprob needs ids")
    if top == 0 and (top_ids is not None and top_ids.numel()
                     or top_logprobs is not None and top_logprobs.numel()):
        raise ValueError("top_ids and top_logprobs need top")
    lpp = _f32(logprob, "logprob", T, at)
    enp = _f32(entropy, "entropy", T, at)
    lsp = _f32(lse, "lse", T, at)
    _workspace_on(ws, at)

    def call(st):
        lp, en, ls, ti, tp, la, ea, sa = logprob, entropy, lse, top_ids, top_logprobs, lpp, enp, lsp
        if lp is None and ids is not None:
            lp = torch.empty(T, dtype=torch.float32, device=z.device)
            la = lp.data_ptr()
        if en is None:
            en = torch.empty(T, dtype=torch.float32, device=z.device)
            ea = en.data_ptr()
        if ls is None:
            ls = torch.empty(T, dtype=torch.float32, device=z.device)
            sa = ls.data_ptr()
        if top > 0:
            if ti is None:
                ti = torch.empty((T, top), dtype=torch.int32, device=z.device)
            if tp is None:
                tp = torch.empty((T, top), dtype=torch.float32, device=z.device)
            tia = _table(ti, "top_ids", T, top, at, torch.int32)
            tpa = _table(tp, "top_logprobs", T, top, at, torch.float32)
        else:
            tia = tpa = None
        w = ws if ws is not None else _workspace(_STATUS_WS, z.device, None)
        rc = (_lib or lib()).token_logprobs(z.data_ptr(), zt, ldz, ip, idb, T, V, scale,
                                            int(padding_idx), top, la, ea, sa,
                                            tia, tpa, w.data_ptr(), w.nbytes, st)
        if rc != OK:
            _check(rc, "token_logprobs")
        return lp, en, ls, ti, tp

    return _at(at, stream, call)


def _grad_rows(out, z, dtype, index):
    """(the tensor, 2-d view, type code, row stride) of a gradient of the logits."""
    if out is None:
        out = torch.empty(z.shape, dtype=dtype or z.dtype, device=z.device)
    elif dtype is not None and out.dtype != dtype:
        raise ValueError("out and out_dtype differ")
    o2, ot, ldo = _rows(out, "the logits' gradient", z.shape[-1], index)[:3]
    if o2.numel() != z.numel():
        raise ValueError("the logits' gradient must have their shape")
    return out, o2, ot, ldo


def token_logprobs_grad(logits, ids, lse, grad_logprob=None, entropy=None, grad_entropy=None,
                        scale=1.0, padding_idx=-1, out=None, out_dtype=None, ws=None, stream=None):
    """Gradient of token_logprobs in the logits: scale (grad_logprob (1[i = id] - p_i)
    - grad_entropy p_i (log p_i + entropy)) of each row, in the logits' type by
    default.  lse, entropy: token_logprobs'; grad_logprob, grad_entropy: float32
    [rows] or None for 0 (entropy is needed with the latter).  out may be the
    logits.  Rows that are padding or whose gradients are 0 are not read and
    give zeros."""
    z, zt, ldz, at, T, V = _rows(logits, "logits")
    ip, idb = (None, 8) if ids is None else _id_list(ids, "ids", T, at)
    if lse is None or (grad_entropy is not None and entropy is None) or \
            (grad_logprob is not None and ids is None):
        raise ValueError("lse, ids for grad_logprob and entropy for grad_entropy are needed")
    sp = _f32(lse, "lse", T, at)
    ep = _f32(entropy, "entropy", T, at)
    gp = _f32(grad_logprob, "grad_logprob", T, at)
    hp = _f32(grad_entropy, "grad_entropy", T, at)
    _workspace_on(ws, at)

    def call(st):
        o, o2, ot, ldo = _grad_rows(out, logits, out_dtype, at)
        w = ws if ws is not None else _workspace(_STATUS_WS, z.device, None)
        rc = (_lib or lib()).token_logprobs_grad(z.data_ptr(), zt, ldz, ip, idb, T, V, scale,
                                       int(padding_idx), sp, ep, gp, hp, o2.data_ptr(), ot, ldo,
                                       w.data_ptr(), w.nbytes, st)
        if rc != OK:
            _check(rc, "token_logprobs_grad")
        return o

    return _at(at, stream, call)


def distill_loss_workspace_bytes() -> int:
    return int(lib().distill_loss_workspace_bytes())


def distill_loss(logits, teacher_ids, teacher_logits, weight=None, scale=1.0, grad=False, loss=None,
                 grad_logits=None, out_dtype=None, ws=None, stream=None):
    """Distillation from a teacher's top logits: (loss, grad_logits), with
    q = softmax(scale teacher_logits) over the K entries of a row and
    p = softmax(scale logits) over all tokens,
    loss = weight sum_k q_k (log q_k - log p[teacher_ids_k]), float32 [rows], and the
    gradient of its sum, weight scale (p - q), in the logits' type by default:
    with grad or a grad_logits to write (which may be the logits), else None.
    teacher_ids: int32 / int64 [rows, K] (token_logprobs' top_ids; negative: no
    entry); teacher_logits: [rows, K]; weight: float32 [rows] or None for 1.  An id
    past V gives ERR_BAD_INPUT from topk_ef_last_device_status(ws) and counts
    nowhere."""
    z, zt, ldz, at, T, V = _rows(logits, "logits")
    shape = teacher_ids.shape if isinstance(teacher_ids, torch.Tensor) else ()
    if not shape:
        raise ValueError("teacher_ids must be [rows, K]")
    K = shape[-1]
    ip, idb = _id_list(teacher_ids, "teacher_ids", T * K, at)
    tp, tt = _vector(teacher_logits, "teacher_logits", T * K, at)
    if tp is None:
        raise ValueError("teacher_logits are needed")
    if teacher_logits.shape != shape and teacher_logits.shape[-1:] != shape[-1:]:
        raise ValueError(f"teacher_logits must be [{T}, {K}]")
    wp = _f32(weight, "weight", T, at)
    lp = _f32(loss, "loss", T, at)
    _workspace_on(ws, at)

    def call(st):
        lo, la, o, op, ot, ldo = loss, lp, grad_logits, None, 0, V
        if lo is None:
            lo = torch.empty(T, dtype=torch.float32, device=z.device)
            la = lo.data_ptr()
        if grad or o is not None:
            o, o2, ot, ldo = _grad_rows(o, logits, out_dtype, at)
            op = o2.data_ptr()
        w = ws if ws is not None else _workspace(_STATUS_WS, z.device, None)
        rc = (_lib or lib()).distill_loss(z.data_ptr(), zt, ldz, ip, idb, tp, tt,
                                          T, V, K, scale, wp, la, op, ot, ldo, w.data_ptr(),
                                          w.nbytes, st)
        if rc != OK:
            _check(rc, "distill_loss")
        return lo, o

    return _at(at, stream, call)


# -------------------------------------------------------------------- status

def topk_ef_last_device_status(ws, stream=None) -> int:
    return int(lib().topk_ef_last_device_status(ws.data_ptr(), _stream(stream)))


def topk_ef_path_info(ws, stream=None) -> dict:
    info = (ctypes.c_int64 * 6)()
    _check(lib().topk_ef_path_info(ws.data_ptr(), _stream(stream), info), "topk_ef_path_info")
    return {"fallback": int(info[0]), "candidates": int(info[1]), "capacity": int(info[2]),
            "kernels": int(info[3]), "crowded_bin": int(info[4])}


def topk_ef_phase_times(ws, stream=None) -> list:
    """Diagnostic timestamps of the last compress call on ws (20 values, ns;
    -1: step not run): select kernel phases, the sampling block, then the
    streaming and select kernels' spans over all blocks."""
    ns = (ctypes.c_int64 * 20)()
    _check(lib().topk_ef_phase_times(ws.data_ptr(), _stream(stream), ns), "topk_ef_phase_times")
    return [int(x) for x in ns]


def topk_ef_set_test_flags(flags: int) -> int:
    return int(lib().topk_ef_set_test_flags(int(flags)))


def topk_ef_trace_enable(on: bool = True, only: str | None = None, every: int = 1) -> None:
    """Record CUDA events around every kernel the library launches, or only
    around the launches of kernel `only`, every `every`-th of them."""
    L = lib()
    _check(L.topk_ef_trace_only(only.encode() if only else None, int(every)),
           "topk_ef_trace_only")
    _check(L.topk_ef_trace_enable(1 if on else 0), "topk_ef_trace_enable")


def topk_ef_trace_read() -> list:
    """[(kernel name, milliseconds)] of the launches recorded since tracing
    was enabled or last read (waits for them to finish), and clears them."""
    ms = (ctypes.c_float * 4096)()
    names = (ctypes.c_char_p * 4096)()
    cnt = ctypes.c_int(0)
    _check(lib().topk_ef_trace_read(ms, names, 4096, ctypes.byref(cnt)), "topk_ef_trace_read")
    return [(names[i].decode(), float(ms[i])) for i in range(cnt.value)]
