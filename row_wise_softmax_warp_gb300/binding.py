"""Python binding of librowops (include/rowops.h): argument marshalling only.

Every function has the name of its C entry point, takes torch CUDA tensors
(fp32, contiguous, last dimension = cols, rows = numel / cols), allocates the
outputs the caller leaves as ``None`` with torch, passes raw device pointers
and the current torch stream to the C ABI and raises ``RowopsError`` on a
nonzero status.  All arithmetic happens in the library's CUDA kernels; there
is no other code path.  The library is loaded on first use and a missing build
is an error, never a fallback.
"""
from __future__ import annotations

import ctypes
import math
import os

import torch

LIB_PATH = os.path.join(os.path.dirname(os.path.abspath(__file__)), "librowops.so")

_lib = None

_P = ctypes.c_void_p
_I64 = ctypes.c_int64
_F = ctypes.c_float
_I = ctypes.c_int

SIGNATURES = {
    "rowops_status_string": ([ctypes.c_int], ctypes.c_char_p),
    "rowops_kernel_launches": ([], ctypes.c_uint64),
    "rowops_pipeline_timeouts": ([], ctypes.c_uint32),
    "rowops_softmax_fwd": ([_P, _P, _I64, _I64, _P], ctypes.c_int),
    "rowops_softmax_bwd": ([_P, _P, _P, _I64, _I64, _P], ctypes.c_int),
    "rowops_attn_softmax_fwd": ([_P, _P, _I64, _I64, _I64, _F, _P], ctypes.c_int),
    "rowops_attn_softmax_bwd": ([_P, _P, _P, _I64, _I64, _I64, _F, _P], ctypes.c_int),
    "rowops_masked_softmax": ([_P, _P, _P, _I64, _I64, _P], ctypes.c_int),
    "rowops_logsumexp": ([_P, _P, _I64, _I64, _P], ctypes.c_int),
    "rowops_softmax_ce": ([_P, _P, _P, _P, _P, _I64, _I64, _F, _P], ctypes.c_int),
    "rowops_layernorm_fwd": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _F, _P], ctypes.c_int),
    "rowops_layernorm_bwd_workspace": ([_I64, _I64], ctypes.c_size_t),
    "rowops_layernorm_bwd": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _P, ctypes.c_size_t, _P],
                             ctypes.c_int),
    "rowops_topk_kept": ([_P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "rowops_router_masked_topk": ([_P, _P, _P, _P, _I64, _I64, _I64, _P], ctypes.c_int),
    "rowops_top_k_rows": ([_P, _P, _P, _I64, _I64, _I64, ctypes.c_int, _P], ctypes.c_int),
    "rowops_rmsnorm_fwd": ([_P, _P, _P, _P, _I64, _I64, _F, _P], ctypes.c_int),
    "rowops_rmsnorm_bwd": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _P], ctypes.c_int),
    "rowops_column_sums": ([_P, _P, _I64, _I64, _F, _P], ctypes.c_int),
    "rowops_masked_softmax_fmask": ([_P, _P, _P, _I64, _I64, _P], ctypes.c_int),
    "rowops_lrp_softmax_rows": ([_P, _P, _P, _P, _I64, _I64, _P], ctypes.c_int),
    "rowops_argmax_onehot": ([_P, _P, _I64, _I64, _P], ctypes.c_int),
    "rowops_soft_ce": ([_P, _P, _P, _P, _P, _I64, _I64, _F, _P], ctypes.c_int),
    "rowops_teacher_ce": ([_P, _P, _P, _P, _P, _I64, _I64, _F, _P], ctypes.c_int),
    "rowops_layernorm_bwd_noalloc": ([_P, _P, _P, _P, _P, _P, _P, _I64, _I64, _P], ctypes.c_int),
    "rowops_layernorm_bwd_noalloc_max_bytes": ([], ctypes.c_size_t),
    "rowops_expert_plan_workspace": ([_I64, _I64, _I64], ctypes.c_size_t),
    "rowops_expert_plan": ([_P, _P, _P, _P, _P, _I64, _I64, _I64, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "rowops_expert_gather": ([_P, _P, _P, _I64, _I64, _I64, _I64, _I, _I, _P], ctypes.c_int),
    "rowops_expert_combine": ([_P, _P, _P, _P, _I64, _I64, _I64, _I64, _I, _I, _P], ctypes.c_int),
    "rowops_expert_combine_bwd": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I, _I, _P], ctypes.c_int),
    "rowops_expert_matmul": ([_P, _P, _P, _P, _I64, _I64, _I64, _I64, _I, _I, _P, ctypes.c_size_t, _P], ctypes.c_int),
    "rowops_expert_matmul_workspace": ([_I64, _I64, _I64, _I64, _I], ctypes.c_size_t),
    "rowops_expert_matmul_wgrad": ([_P, _P, _P, _P, _I64, _I64, _I64, _I64, _I, _I, _P, ctypes.c_size_t, _P],
                                   ctypes.c_int),
    "rowops_expert_matmul_wgrad_workspace": ([_I64, _I64, _I64], ctypes.c_size_t),
    "rowops_expert_matmul_fp8_workspace": ([_I64, _I64, _I64, _I64], ctypes.c_size_t),
    "rowops_quantize_blocks": ([_P, _P, _P, _I64, _I64, _I64, _I64, _I, _P], ctypes.c_int),
    "rowops_expert_matmul_fp8": ([_P, _P, _P, _P, _P, _P, _I64, _I64, _I64, _I64, _I, _P, ctypes.c_size_t, _P],
                                 ctypes.c_int),
}


class RowopsError(RuntimeError):
    """A rowops_* entry point returned a nonzero status."""

    def __init__(self, status: int, message: str):
        super().__init__(message)
        self.status = status


def library():
    """The loaded librowops (ctypes.CDLL) with its C signatures declared."""
    global _lib
    if _lib is None:
        if not os.path.exists(LIB_PATH):
            raise RuntimeError(
                f"{LIB_PATH} is missing: build it with row_wise_softmax_warp_gb300.build.build() "
                "(or __graft_entry__.build()); there is no fallback implementation")
        lib = ctypes.CDLL(LIB_PATH)
        for name, (args, res) in SIGNATURES.items():
            fn = getattr(lib, name)
            fn.argtypes = args
            fn.restype = res
        _lib = lib
    return _lib


def _check(status: int):
    if status != 0:
        raise RowopsError(status, library().rowops_status_string(status).decode())


def _stream(t: torch.Tensor, stream):
    if stream is None:
        return torch.cuda.current_stream(t.device).cuda_stream
    if isinstance(stream, torch.cuda.Stream):
        return stream.cuda_stream
    return int(stream)


def _mat(t: torch.Tensor, name: str, dtype=torch.float32):
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def _shape(t: torch.Tensor):
    if t.dim() == 0:
        return 1, 1
    cols = int(t.shape[-1])
    return math.prod(t.shape[:-1]), cols


def _out(t, like: torch.Tensor, name: str, shape=None, dtype=torch.float32):
    if t is None:
        return torch.empty(like.shape if shape is None else shape, dtype=dtype, device=like.device)
    return _mat(t, name, dtype)


def _bytes_behind(t: torch.Tensor) -> int:
    """Bytes of a workspace: those of its values, but none behind the end of its storage (an expanded view names
    more values than it holds)."""
    size = t.element_size()
    return min(t.numel() * size, t.untyped_storage().nbytes() - t.storage_offset() * size)


def rowops_kernel_launches() -> int:
    return int(library().rowops_kernel_launches())


def rowops_softmax_fwd(x, y=None, stream=None):
    """y = softmax(x) along the last dimension (y may be x)."""
    x = _mat(x, "x")
    y = _out(y, x, "y")
    rows, cols = _shape(x)
    _check(library().rowops_softmax_fwd(x.data_ptr(), y.data_ptr(), rows, cols, _stream(x, stream)))
    return y


def rowops_softmax_bwd(y, dy, dx=None, stream=None):
    """dx = y * (dy - sum(y * dy)) along the last dimension."""
    y, dy = _mat(y, "y"), _mat(dy, "dy")
    dx = _out(dx, y, "dx")
    rows, cols = _shape(y)
    _check(library().rowops_softmax_bwd(y.data_ptr(), dy.data_ptr(), dx.data_ptr(), rows, cols,
                                        _stream(y, stream)))
    return dx


def rowops_attn_softmax_fwd(scores, p=None, seq_len=None, scale=1.0, stream=None):
    """Scaled causal softmax of stacked (batch*heads*seq_len, seq_len) score rows."""
    scores = _mat(scores, "scores")
    p = _out(p, scores, "p")
    rows, cols = _shape(scores)
    seq_len = cols if seq_len is None else seq_len
    _check(library().rowops_attn_softmax_fwd(scores.data_ptr(), p.data_ptr(), rows, cols, seq_len,
                                             scale, _stream(scores, stream)))
    return p


def rowops_attn_softmax_bwd(p, dp, ds=None, seq_len=None, scale=1.0, stream=None):
    """Gradient of rowops_attn_softmax_fwd with respect to the raw scores, from p."""
    p, dp = _mat(p, "p"), _mat(dp, "dp")
    ds = _out(ds, p, "ds")
    rows, cols = _shape(p)
    seq_len = cols if seq_len is None else seq_len
    _check(library().rowops_attn_softmax_bwd(p.data_ptr(), dp.data_ptr(), ds.data_ptr(), rows, cols,
                                             seq_len, scale, _stream(p, stream)))
    return ds


def rowops_masked_softmax(x, mask, y=None, stream=None):
    """Softmax over entries with mask != 0; blocked entries and empty rows are +0."""
    x = _mat(x, "x")
    mask = _mat(mask, "mask", torch.uint8)
    y = _out(y, x, "y")
    rows, cols = _shape(x)
    _check(library().rowops_masked_softmax(x.data_ptr(), mask.data_ptr(), y.data_ptr(), rows, cols,
                                           _stream(x, stream)))
    return y


def rowops_logsumexp(x, lse=None, stream=None):
    """lse = log(sum(exp(x))) along the last dimension."""
    x = _mat(x, "x")
    rows, cols = _shape(x)
    lse = _out(lse, x, "lse", shape=x.shape[:-1])
    _check(library().rowops_logsumexp(x.data_ptr(), lse.data_ptr(), rows, cols, _stream(x, stream)))
    return lse


def rowops_softmax_ce(logits, targets, grad=None, row_loss=None, mean_loss=None, grad_scale=None,
                      stream=None):
    """Returns (grad, row_loss, mean_loss); mean_loss is a one-element float64 CUDA tensor."""
    logits = _mat(logits, "logits")
    targets = _mat(targets, "targets", torch.int32)
    rows, cols = _shape(logits)
    grad = _out(grad, logits, "grad")
    row_loss = _out(row_loss, logits, "row_loss", shape=(rows,))
    mean_loss = _out(mean_loss, logits, "mean_loss", shape=(1,), dtype=torch.float64)
    if grad_scale is None:
        grad_scale = 1.0 / rows if rows else 1.0
    _check(library().rowops_softmax_ce(logits.data_ptr(), targets.data_ptr(), grad.data_ptr(),
                                       row_loss.data_ptr(), mean_loss.data_ptr(), rows, cols,
                                       grad_scale, _stream(logits, stream)))
    return grad, row_loss, mean_loss


def rowops_layernorm_fwd(x, gamma, beta, out=None, xhat=None, inv_std=None, eps=1e-5, stream=None):
    """Returns (out, xhat, inv_std)."""
    x, gamma, beta = _mat(x, "x"), _mat(gamma, "gamma"), _mat(beta, "beta")
    rows, cols = _shape(x)
    out = _out(out, x, "out")
    xhat = _out(xhat, x, "xhat")
    inv_std = _out(inv_std, x, "inv_std", shape=(rows,))
    _check(library().rowops_layernorm_fwd(x.data_ptr(), gamma.data_ptr(), beta.data_ptr(),
                                          out.data_ptr(), xhat.data_ptr(), inv_std.data_ptr(), rows,
                                          cols, eps, _stream(x, stream)))
    return out, xhat, inv_std


def rowops_layernorm_bwd_workspace(rows: int, cols: int) -> int:
    return int(library().rowops_layernorm_bwd_workspace(rows, cols))


def rowops_layernorm_bwd(dy, gamma, xhat, inv_std, dx=None, dgamma=None, dbeta=None, workspace=None,
                         stream=None):
    """Returns (dx, dgamma, dbeta)."""
    dy, gamma, xhat = _mat(dy, "dy"), _mat(gamma, "gamma"), _mat(xhat, "xhat")
    inv_std = _mat(inv_std, "inv_std")
    rows, cols = _shape(dy)
    dx = _out(dx, dy, "dx")
    dgamma = _out(dgamma, dy, "dgamma", shape=(cols,))
    dbeta = _out(dbeta, dy, "dbeta", shape=(cols,))
    need = rowops_layernorm_bwd_workspace(rows, cols)
    if workspace is None:
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=dy.device)
    _check(library().rowops_layernorm_bwd(dy.data_ptr(), gamma.data_ptr(), xhat.data_ptr(),
                                          inv_std.data_ptr(), dx.data_ptr(), dgamma.data_ptr(),
                                          dbeta.data_ptr(), rows, cols, workspace.data_ptr(),
                                          _bytes_behind(workspace),
                                          _stream(dy, stream)))
    return dx, dgamma, dbeta


def rowops_topk_kept(x, k, kept=None, stream=None):
    """1.0 where fewer than k entries of the row beat the entry, else 0.0."""
    x = _mat(x, "x")
    kept = _out(kept, x, "kept")
    rows, cols = _shape(x)
    _check(library().rowops_topk_kept(x.data_ptr(), kept.data_ptr(), rows, cols, k,
                                      _stream(x, stream)))
    return kept


def rowops_router_masked_topk(x, mask, k, p=None, kept=None, stream=None):
    """Fused router: returns (p, kept) = (masked softmax of x, top-k kept mask of p)."""
    x = _mat(x, "x")
    mask = _mat(mask, "mask", torch.uint8)
    p = _out(p, x, "p")
    kept = _out(kept, x, "kept")
    rows, cols = _shape(x)
    _check(library().rowops_router_masked_topk(x.data_ptr(), mask.data_ptr(), p.data_ptr(), kept.data_ptr(),
                                               rows, cols, k, _stream(x, stream)))
    return p, kept


def rowops_top_k_rows(x, k, largest=True, values=None, indices=None, stream=None):
    """Returns (values, indices), each (rows, k): the k largest (or smallest) entries
    of every row in rank order (NaN above every number; ties by lower column)."""
    x = _mat(x, "x")
    rows, cols = _shape(x)
    values = _out(values, x, "values", shape=(*x.shape[:-1], k))
    indices = _out(indices, x, "indices", shape=(*x.shape[:-1], k))
    _check(library().rowops_top_k_rows(x.data_ptr(), values.data_ptr(), indices.data_ptr(), rows, cols, k,
                                       1 if largest else 0, _stream(x, stream)))
    return values, indices


def rowops_rmsnorm_fwd(x, gamma, out=None, row_rms=None, eps=1e-5, stream=None):
    """Returns (out, row_rms)."""
    x, gamma = _mat(x, "x"), _mat(gamma, "gamma")
    rows, cols = _shape(x)
    out = _out(out, x, "out")
    row_rms = _out(row_rms, x, "row_rms", shape=(rows,))
    _check(library().rowops_rmsnorm_fwd(x.data_ptr(), gamma.data_ptr(), out.data_ptr(), row_rms.data_ptr(),
                                        rows, cols, eps, _stream(x, stream)))
    return out, row_rms


def rowops_rmsnorm_bwd(dy, gamma, x, row_rms, dx=None, gamma_terms=None, stream=None):
    """Returns (dx, gamma_terms); gamma's gradient is rowops_column_sums(gamma_terms)."""
    dy, gamma, x, row_rms = _mat(dy, "dy"), _mat(gamma, "gamma"), _mat(x, "x"), _mat(row_rms, "row_rms")
    rows, cols = _shape(dy)
    dx = _out(dx, dy, "dx")
    gamma_terms = _out(gamma_terms, dy, "gamma_terms")
    _check(library().rowops_rmsnorm_bwd(dy.data_ptr(), gamma.data_ptr(), x.data_ptr(), row_rms.data_ptr(),
                                        dx.data_ptr(), gamma_terms.data_ptr(), rows, cols, _stream(dy, stream)))
    return dx, gamma_terms


def rowops_column_sums(m, out=None, beta=0.0, stream=None):
    """out_j = beta * out_j + sum_i m_ij (deterministic order)."""
    m = _mat(m, "in")
    rows, cols = _shape(m)
    if out is None:
        out = torch.zeros(cols, dtype=torch.float32, device=m.device)
    out = _mat(out, "out")
    _check(library().rowops_column_sums(m.data_ptr(), out.data_ptr(), rows, cols, beta, _stream(m, stream)))
    return out


def rowops_masked_softmax_fmask(x, mask, y=None, stream=None):
    """Masked softmax with an fp32 mask (allowed where mask != 0)."""
    x, mask = _mat(x, "x"), _mat(mask, "mask")
    y = _out(y, x, "y")
    rows, cols = _shape(x)
    _check(library().rowops_masked_softmax_fmask(x.data_ptr(), mask.data_ptr(), y.data_ptr(), rows, cols,
                                                 _stream(x, stream)))
    return y


def rowops_lrp_softmax_rows(x, y, r, r_in=None, stream=None):
    """r_in = x * (r - y * sum(r)) per row."""
    x, y, r = _mat(x, "x"), _mat(y, "y"), _mat(r, "r")
    r_in = _out(r_in, x, "r_in")
    rows, cols = _shape(x)
    _check(library().rowops_lrp_softmax_rows(x.data_ptr(), y.data_ptr(), r.data_ptr(), r_in.data_ptr(), rows,
                                             cols, _stream(x, stream)))
    return r_in


def rowops_argmax_onehot(x, out=None, stream=None):
    """1.0 at the first maximal coordinate of each row, 0.0 elsewhere."""
    x = _mat(x, "x")
    out = _out(out, x, "out")
    rows, cols = _shape(x)
    _check(library().rowops_argmax_onehot(x.data_ptr(), out.data_ptr(), rows, cols, _stream(x, stream)))
    return out


def _ce2(fn, x, w, grad, row_loss, mean_loss, grad_scale, stream, want_grad=True):
    x, w = _mat(x, "logits"), _mat(w, "weights")
    rows, cols = _shape(x)
    if want_grad:
        grad = _out(grad, x, "grad")
    row_loss = _out(row_loss, x, "row_loss", shape=(rows,))
    mean_loss = _out(mean_loss, x, "mean_loss", shape=(1,), dtype=torch.float64)
    if grad_scale is None:
        grad_scale = 1.0 / rows if rows else 1.0
    _check(fn(x.data_ptr(), w.data_ptr(), grad.data_ptr() if grad is not None else None, row_loss.data_ptr(),
              mean_loss.data_ptr(), rows, cols, grad_scale, _stream(x, stream)))
    return grad, row_loss, mean_loss


def rowops_soft_ce(logits, weights, grad=None, row_loss=None, mean_loss=None, grad_scale=None, stream=None):
    """Weighted-logits (soft-target) CE: returns (grad, row_loss, mean_loss)."""
    return _ce2(library().rowops_soft_ce, logits, weights, grad, row_loss, mean_loss, grad_scale, stream)


def rowops_teacher_ce(student, teacher, grad=None, row_loss=None, mean_loss=None, grad_scale=None,
                      with_grad=True, stream=None):
    """Fixed-teacher CE: returns (student grad or None, row_loss, mean_loss)."""
    return _ce2(library().rowops_teacher_ce, student, teacher, grad, row_loss, mean_loss, grad_scale, stream,
                want_grad=with_grad)


def rowops_layernorm_bwd_noalloc(dy, gamma, xhat, inv_std, dx=None, dgamma=None, dbeta=None, stream=None):
    """rowops_layernorm_bwd without a workspace argument: the library's own
    fixed device array serves as workspace (calls on one device must not
    overlap on the GPU).  Returns (dx, dgamma, dbeta)."""
    dy, gamma, xhat = _mat(dy, "dy"), _mat(gamma, "gamma"), _mat(xhat, "xhat")
    inv_std = _mat(inv_std, "inv_std")
    rows, cols = _shape(dy)
    dx = _out(dx, dy, "dx")
    dgamma = _out(dgamma, dy, "dgamma", shape=(cols,))
    dbeta = _out(dbeta, dy, "dbeta", shape=(cols,))
    _check(library().rowops_layernorm_bwd_noalloc(dy.data_ptr(), gamma.data_ptr(), xhat.data_ptr(),
                                                  inv_std.data_ptr(), dx.data_ptr(), dgamma.data_ptr(),
                                                  dbeta.data_ptr(), rows, cols, _stream(dy, stream)))
    return dx, dgamma, dbeta


# ------------------------------------------------------- the expert operators
# Outputs left as ``None`` and workspaces are allocated on the call's stream.  A
# small call takes the device a few microseconds, so arguments that are as they
# should be pass one short test each; what is wrong is found out afterwards.

_DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}  # rowops_dtype
_FLOATS = (torch.float32, torch.float16, torch.bfloat16)
_HALVES = (torch.float16, torch.bfloat16)
_F32 = (torch.float32,)
_INT = (torch.int32,)
_E4M3 = (torch.float8_e4m3fn,)
_ONE_LAUNCH_PAIRS = 2048  # plans of so many pairs need no workspace, as the header says


class _Placed:
    """Makes a tensor's device, and a stream if one is given, current for allocations and the launch."""

    def __init__(self, t: torch.Tensor, stream):
        device = getattr(stream, "device", None)  # a handle does not say
        if device is not None and device != t.device:
            raise ValueError(f"stream is on {device}, the tensors are on {t.device}")
        self.guards = [torch.cuda.device(t.device)]
        if stream is not None:
            if not isinstance(stream, torch.cuda.Stream):
                stream = (torch.cuda.ExternalStream(int(stream), device=t.device) if int(stream)
                          else torch.cuda.default_stream(t.device))
            self.guards.append(torch.cuda.stream(stream))

    def __enter__(self):
        for g in self.guards:
            g.__enter__()

    def __exit__(self, *exc):
        for g in reversed(self.guards):
            g.__exit__(*exc)


def _elsewhere(t, stream) -> bool:
    """Whether the call has to make another device or stream current first."""
    return stream is not None or t.get_device() != _current_device()


def _typed(t, name: str, dtypes, shape=None, device=None):
    """A contiguous CUDA tensor of one of `dtypes`, of `shape` and on device number `device` where they are given."""
    if (isinstance(t, torch.Tensor) and t.is_cuda and t.dtype in dtypes and t.is_contiguous()
            and (shape is None or t.shape == shape) and (device is None or t.get_device() == device)):
        return t
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise TypeError(f"{name} must be a CUDA tensor")
    if t.dtype not in dtypes:
        raise TypeError(f"{name} must be {' or '.join(str(d) for d in dtypes)}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and t.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    raise ValueError(f"{name} is on cuda:{t.get_device()}, not on cuda:{device}")


def _dims(t, name: str, n: int):
    shape = t.shape
    if len(shape) != n:
        raise ValueError(f"{name} must have {n} dimensions, got {len(shape)}")
    return shape


def _given(t, name: str, dtype, shape, like, device):
    """An output: the caller's, checked, or a new one."""
    if t is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    return _typed(t, name, (dtype,), shape, device)


def _scratch(workspace, need: int, like):
    """(workspace, its bytes): the caller's, or a new one of `need` bytes where that is not 0."""
    if workspace is not None:
        if not isinstance(workspace, torch.Tensor) or workspace.device != like.device:
            raise ValueError(f"workspace must be a tensor on {like.device}")
        if not workspace.is_contiguous():  # its bytes are counted from its values
            raise ValueError("workspace must be contiguous")
        return workspace, workspace.numel() * workspace.element_size()
    return (torch.empty(need, dtype=torch.uint8, device=like.device), need) if need else (None, 0)


def _shifted_room(*operands) -> int:
    """Bytes for copies of the matrices (tensor, rows, bytes of a row) that start off a 16-byte boundary; the
    workspace functions of the library see only the widths, and count rows that are no multiple of 16 bytes."""
    return sum(rows * size + 512 for t, rows, size in operands if t.data_ptr() % 16 and size % 16 == 0)


def _ptr(t):
    return None if t is None else t.data_ptr()


# t is a CUDA tensor, so CUDA is initialised
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda device: torch.cuda.current_stream(device).cuda_stream)


def rowops_expert_plan_workspace(rows: int, k: int, experts: int) -> int:
    return int(library().rowops_expert_plan_workspace(rows, k, experts))


def rowops_expert_plan(indices, experts, values=None, offsets=None, order=None, slot=None, workspace=None,
                       stream=None):
    """Returns (offsets, order, slot), int32: the (token, choice) pairs of indices (rows, k) grouped by expert.

    values (rows, k): pairs whose value is 0 are left out."""
    _typed(indices, "indices", _F32)
    if _elsewhere(indices, stream):
        with _Placed(indices, stream):
            return rowops_expert_plan(indices, experts, values, offsets, order, slot, workspace)
    rows, k = shape = _dims(indices, "indices", 2)
    device = indices.get_device()
    if values is not None:
        _typed(values, "values", _F32, shape, device)
    lib = library()
    pairs = rows * k
    need = lib.rowops_expert_plan_workspace(rows, k, experts) if workspace is None and pairs > _ONE_LAUNCH_PAIRS else 0
    offsets = _given(offsets, "offsets", torch.int32, (max(experts, 0) + 1,), indices, device)
    order = _given(order, "order", torch.int32, (pairs,), indices, device)
    slot = _given(slot, "slot", torch.int32, shape, indices, device)
    workspace, size = _scratch(workspace, need, indices)
    _check(lib.rowops_expert_plan(indices.data_ptr(), _ptr(values), offsets.data_ptr(), order.data_ptr(),
                                  slot.data_ptr(), rows, k, experts, _ptr(workspace), size, _raw_stream(device)))
    return offsets, order, slot


def rowops_expert_gather(x, slot, out=None, slots=None, dtype=None, stream=None):
    """out[slot[t][j]] = x[t]; x (rows, cols), slot (rows, k).  A new `out` has `slots` rows (default rows * k)
    of `dtype` (default x's); its rows that no slot names are not written."""
    _typed(x, "x", _FLOATS)
    if _elsewhere(x, stream):
        with _Placed(x, stream):
            return rowops_expert_gather(x, slot, out, slots, dtype)
    rows, cols = _dims(x, "x", 2)
    device = x.get_device()
    k = _dims(_typed(slot, "slot", _INT, None, device), "slot", 2)[1]
    if slot.shape[0] != rows:
        raise ValueError(f"slot must have {rows} rows, got {slot.shape[0]}")
    if out is None:
        out = torch.empty((rows * k if slots is None else slots, cols), dtype=x.dtype if dtype is None else dtype,
                          device=x.device)
    _typed(out, "out", _FLOATS if dtype is None else (dtype,), None, device)
    if len(out.shape) != 2 or out.shape[1] != cols or (slots is not None and out.shape[0] != slots):
        raise ValueError(f"out must have shape ({'slots' if slots is None else slots}, {cols}), got {tuple(out.shape)}")
    _check(library().rowops_expert_gather(x.data_ptr(), slot.data_ptr(), out.data_ptr(), rows, k, cols, out.shape[0],
                                          _DTYPES[x.dtype], _DTYPES.get(out.dtype, -1), _raw_stream(device)))
    return out


def rowops_expert_combine(y, slot, weights=None, out=None, dtype=None, stream=None):
    """out[t] = sum_j weights[t][j] * y[slot[t][j]] (weights None: all 1); out of `dtype` (default y's)."""
    _typed(y, "y", _FLOATS)
    if _elsewhere(y, stream):
        with _Placed(y, stream):
            return rowops_expert_combine(y, slot, weights, out, dtype)
    slots, cols = _dims(y, "y", 2)
    device = y.get_device()
    rows, k = pairs = _dims(_typed(slot, "slot", _INT, None, device), "slot", 2)
    if weights is not None:
        _typed(weights, "weights", _F32, pairs, device)
    if out is None:
        out = torch.empty((rows, cols), dtype=y.dtype if dtype is None else dtype, device=y.device)
    else:
        _typed(out, "out", _FLOATS if dtype is None else (dtype,), (rows, cols), device)
    _check(library().rowops_expert_combine(y.data_ptr(), slot.data_ptr(), _ptr(weights), out.data_ptr(), rows, k, cols,
                                           slots, _DTYPES[y.dtype], _DTYPES.get(out.dtype, -1), _raw_stream(device)))
    return out


def rowops_expert_combine_bwd(dout, y, slot, weights, dy=None, dweights=None, stream=None):
    """Returns (dy, dweights) of rowops_expert_combine; rows of a new dy that no slot names are not written."""
    _typed(y, "y", _FLOATS)
    if _elsewhere(y, stream):
        with _Placed(y, stream):
            return rowops_expert_combine_bwd(dout, y, slot, weights, dy, dweights)
    slots, cols = shape = _dims(y, "y", 2)
    device = y.get_device()
    rows, k = pairs = _dims(_typed(slot, "slot", _INT, None, device), "slot", 2)
    _typed(dout, "dout", _FLOATS, (rows, cols), device)
    _typed(weights, "weights", _F32, pairs, device)
    dy = _given(dy, "dy", y.dtype, shape, y, device)
    dweights = _given(dweights, "dweights", torch.float32, pairs, y, device)
    _check(library().rowops_expert_combine_bwd(dout.data_ptr(), y.data_ptr(), slot.data_ptr(), weights.data_ptr(),
                                               dy.data_ptr(), dweights.data_ptr(), rows, k, cols, slots,
                                               _DTYPES[dout.dtype], _DTYPES[y.dtype], _raw_stream(device)))
    return dy, dweights


def _offsets(offsets, experts: int, device):
    if offsets is not None:
        _typed(offsets, "offsets", _INT, (experts + 1,), device)
    elif experts != 1:
        raise ValueError("offsets may be None for one expert only")


def rowops_expert_matmul_workspace(slots: int, in_cols: int, out_cols: int, experts: int, transposed=False) -> int:
    return int(library().rowops_expert_matmul_workspace(slots, in_cols, out_cols, experts, 1 if transposed else 0))


def rowops_expert_matmul_wgrad_workspace(slots: int, in_cols: int, out_cols: int) -> int:
    return int(library().rowops_expert_matmul_wgrad_workspace(slots, in_cols, out_cols))


def rowops_expert_matmul_fp8_workspace(slots: int, in_cols: int, out_cols: int, experts: int) -> int:
    return int(library().rowops_expert_matmul_fp8_workspace(slots, in_cols, out_cols, experts))


def rowops_expert_matmul(x, w, offsets=None, y=None, transposed=False, workspace=None, stream=None):
    """y[s] = w[e] @ x[s] for the rows offsets[e] <= s < offsets[e + 1] of x (slots, in).

    w: (experts, out, in), or (experts, in, out) with transposed.  Rows of a new y that no expert has are not written.
    A workspace (one is made where it is None) takes copies of matrices whose rows are no multiple of 16 bytes or
    that start off a 16-byte boundary."""
    _typed(x, "x", _HALVES)
    if _elsewhere(x, stream):
        with _Placed(x, stream):
            return rowops_expert_matmul(x, w, offsets, y, transposed, workspace)
    slots, in_cols = _dims(x, "x", 2)
    device, dtype = x.get_device(), x.dtype
    experts, out_cols, k = _dims(_typed(w, "w", (dtype,), None, device), "w", 3)
    if transposed:
        out_cols, k = k, out_cols
    if k != in_cols:
        raise ValueError(f"w must take rows of {in_cols} values, got {tuple(w.shape)}")
    _offsets(offsets, experts, device)
    y = _given(y, "y", dtype, (slots, out_cols), x, device)
    lib, flag = library(), 1 if transposed else 0
    need = 0 if in_cols % 8 == 0 and out_cols % 8 == 0 else lib.rowops_expert_matmul_workspace(
        slots, in_cols, out_cols, experts, flag)
    if (x.data_ptr() | w.data_ptr()) % 16 and workspace is None:
        need += _shifted_room((x, slots, 2 * in_cols), (w, experts * w.shape[1], 2 * w.shape[2]))
    workspace, size = _scratch(workspace, need, x)
    _check(lib.rowops_expert_matmul(x.data_ptr(), w.data_ptr(), _ptr(offsets), y.data_ptr(), slots, in_cols, out_cols,
                                    experts, flag, _DTYPES[dtype], _ptr(workspace), size, _raw_stream(device)))
    return y


def rowops_expert_matmul_wgrad(dy, x, offsets=None, dw=None, dtype=None, workspace=None, stream=None):
    """dw[e] = sum over expert e's rows of dy[s]^T x[s]: (experts, out, in), of x's type or torch.float32."""
    _typed(dy, "dy", _HALVES)
    if _elsewhere(dy, stream):
        with _Placed(dy, stream):
            return rowops_expert_matmul_wgrad(dy, x, offsets, dw, dtype, workspace)
    slots, out_cols = _dims(dy, "dy", 2)
    device = dy.get_device()
    in_cols = _dims(_typed(x, "x", (dy.dtype,), None, device), "x", 2)[1]
    if x.shape[0] != slots:
        raise ValueError(f"x must have {slots} rows, got {x.shape[0]}")
    experts = 1
    if offsets is not None:
        experts = _typed(offsets, "offsets", _INT, None, device).numel() - 1
        _offsets(offsets, experts, device)
    shape = (max(experts, 0), out_cols, in_cols)
    if dw is None:
        dw = torch.empty(shape, dtype=dy.dtype if dtype is None else dtype, device=dy.device)
    else:
        _typed(dw, "dw", (dy.dtype, torch.float32) if dtype is None else (dtype,), shape, device)
    lib = library()
    need = lib.rowops_expert_matmul_wgrad_workspace(slots, in_cols, out_cols)
    if (dy.data_ptr() | x.data_ptr()) % 16 and workspace is None:
        need += _shifted_room((dy, slots, 2 * out_cols), (x, slots, 2 * in_cols))
    workspace, size = _scratch(workspace, need, dy)
    _check(lib.rowops_expert_matmul_wgrad(dy.data_ptr(), x.data_ptr(), _ptr(offsets), dw.data_ptr(), slots, in_cols,
                                          out_cols, experts, _DTYPES[dy.dtype], _DTYPES.get(dw.dtype, -1),
                                          _ptr(workspace), size, _raw_stream(device)))
    return dw


def rowops_quantize_blocks(x, block_rows=1, q=None, scale=None, stream=None):
    """Returns (q, scale): e4m3 values of x (..., rows, cols) and an fp32 scale for each block of
    block_rows (1 or 128) rows by 128 columns, scale: (..., ceil(rows / block_rows), ceil(cols / 128))."""
    _typed(x, "x", _FLOATS)
    if _elsewhere(x, stream):
        with _Placed(x, stream):
            return rowops_quantize_blocks(x, block_rows, q, scale)
    shape = x.shape
    if len(shape) < 2:
        raise ValueError("x must have rows and columns")
    if block_rows != 1 and block_rows != 128:
        raise ValueError("block_rows must be 1 or 128")
    rows, cols = shape[-2:]
    device = x.get_device()
    q = _given(q, "q", torch.float8_e4m3fn, shape, x, device)
    scale = _given(scale, "scale", torch.float32, (*shape[:-2], -(-rows // block_rows), -(-cols // 128)), x, device)
    _check(library().rowops_quantize_blocks(x.data_ptr(), q.data_ptr(), scale.data_ptr(), math.prod(shape[:-2]), rows,
                                            cols, block_rows, _DTYPES[x.dtype], _raw_stream(device)))
    return q, scale


def rowops_expert_matmul_fp8(xq, xs, wq, ws, offsets=None, y=None, dtype=torch.bfloat16, workspace=None, stream=None):
    """rowops_expert_matmul on e4m3 operands: xq (slots, in) with xs, wq (experts, out, in) with ws, as
    rowops_quantize_blocks gives them with block_rows 1 and 128; y of `dtype`."""
    _typed(xq, "xq", _E4M3)
    if _elsewhere(xq, stream):
        with _Placed(xq, stream):
            return rowops_expert_matmul_fp8(xq, xs, wq, ws, offsets, y, dtype, workspace)
    slots, in_cols = _dims(xq, "xq", 2)
    device = xq.get_device()
    experts, out_cols, k = _dims(_typed(wq, "wq", _E4M3, None, device), "wq", 3)
    if k != in_cols:
        raise ValueError(f"wq must take rows of {in_cols} values, got {tuple(wq.shape)}")
    blocks = -(-in_cols // 128)
    _typed(xs, "xs", _F32, (slots, blocks), device)
    _typed(ws, "ws", _F32, (experts, -(-out_cols // 128), blocks), device)
    _offsets(offsets, experts, device)
    if y is None:
        y = torch.empty((slots, out_cols), dtype=dtype, device=xq.device)
    else:
        _typed(y, "y", _FLOATS, (slots, out_cols), device)
    lib = library()
    need = lib.rowops_expert_matmul_fp8_workspace(slots, in_cols, out_cols, experts)
    if (xq.data_ptr() | wq.data_ptr()) % 16 and workspace is None:
        need += _shifted_room((xq, slots, in_cols), (wq, experts * out_cols, in_cols))
    workspace, size = _scratch(workspace, need, xq)
    _check(lib.rowops_expert_matmul_fp8(xq.data_ptr(), xs.data_ptr(), wq.data_ptr(), ws.data_ptr(), _ptr(offsets),
                                        y.data_ptr(), slots, in_cols, out_cols, experts, _DTYPES.get(y.dtype, -1),
                                        _ptr(workspace), size, _raw_stream(device)))
    return y
