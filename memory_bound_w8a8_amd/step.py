"""Binding of the operators of include/fp8bq_step.h: the norm in front of the
linear layer with its 8-bit output, the linear layer in 8-bit integers, and
the verification of drafted tokens.

    a_q, a_s, h = rmsnorm_quant(x, weight, residual)       # -> gemm(a_q, a_s, ...)
    a_q, a_s, h = rmsnorm_quant_i8(x, weight, residual)    # -> gemm_i8(a_q, a_s, ...)
    w_q, w_s = quant_weight_i8(w)
    c = gemm_i8(a_q, a_s, w_q, w_s)
    tokens, accepted = verify_drafts(target_p, drafts, u_accept, u_sample, draft_p)

Argument marshalling only, as in the package itself: tensors are checked,
outputs allocated, and the call enqueued on the current stream of the
tensors' device. Calls whose arguments are in order go through _binding.so
(csrc/binding.cpp), which does all of it in one step; what it does not take
comes back to the Python below, which raises, or calls on another device. Where
_binding.so has not been built, that Python makes every call, about 4 us slower
on the host.
"""

import ctypes
import warnings

import torch

from . import Fp8bqError, _check, _need, lib

# Every symbol include/fp8bq_step.h declares.
STEP_EXPORTS = (
    "fp8bq_rmsnorm_quant",
    "fp8bq_rmsnorm_quant_i8",
    "fp8bq_quant_act_i8",
    "fp8bq_quant_weight_i8",
    "fp8bq_gemm_i8_workspace_bytes",
    "fp8bq_gemm_i8",
    "fp8bq_verify_workspace_bytes",
    "fp8bq_verify_drafts",
)

NORM_MAX_K = 65536
GEMM_I8_MAX_K = 130944
MAX_DRAFTS = 64
F32, BF16 = 0, 1

_calls = None


def step_lib():
    """libfp8bq.so with the argument types of this header's calls set."""
    global _calls
    if _calls is None:
        L = lib()
        i64, vp, ci, dbl = ctypes.c_int64, ctypes.c_void_p, ctypes.c_int, ctypes.c_double
        L.fp8bq_rmsnorm_quant.argtypes = [i64, i64, vp, vp, vp, dbl, vp, vp, vp, vp]
        L.fp8bq_rmsnorm_quant_i8.argtypes = [i64, i64, vp, vp, vp, dbl, vp, vp, vp, vp]
        L.fp8bq_quant_act_i8.argtypes = [i64, i64, vp, vp, vp, vp]
        L.fp8bq_quant_weight_i8.argtypes = [i64, i64, vp, vp, vp, vp]
        L.fp8bq_gemm_i8_workspace_bytes.argtypes = [i64, i64, i64]
        L.fp8bq_gemm_i8.argtypes = [i64, i64, i64, vp, vp, vp, vp, vp, vp, i64, vp]
        L.fp8bq_verify_workspace_bytes.argtypes = [i64, i64, i64]
        L.fp8bq_verify_drafts.argtypes = [i64, i64, i64, ci, vp, vp, vp, vp, vp, vp, vp, i64, vp, vp, vp]
        for name in STEP_EXPORTS:
            getattr(L, name).restype = i64 if name.endswith("_bytes") else ci
        _calls = L
    return _calls


_raw_stream = torch._C._cuda_getCurrentRawStream  # 0.1 us; a Stream object takes 2.7
_device = torch._C._cuda_getDevice
_direct = None


class _NoBinding:
    """In the place of _binding.so: leaves every call to Python."""

    @staticmethod
    def rmsnorm(*args):
        return None

    gemm_i8 = verify_drafts = rmsnorm


def _binding(first):
    """The module _binding.so, or _NoBinding (raises if there is no GPU that the
    call's first tensor could be on)."""
    global _direct
    if _direct is None:
        step_lib()
        if not torch.cuda.is_available():
            if not isinstance(first, torch.Tensor):
                raise TypeError("expected torch.Tensors")
            raise ValueError(f"tensors must be on a GPU, got one on {first.device}")
        torch.cuda.init()
        try:
            from . import _binding as module
        except ImportError as e:
            warnings.warn(f"_binding.so is missing or does not load ({e}): calls take the longer way through ctypes; "
                          "build it with `python -m memory_bound_w8a8_amd.build`", RuntimeWarning)
            module = _NoBinding
        _direct = module
    return _direct


def _done(call, out):
    """`out` of a _binding call, None where the call was left to Python."""
    if out.__class__ is int:
        raise Fp8bqError(call, out)
    return out


_empty, _empty_like = torch.empty, torch.empty_like
_BF16, _F32, _I32, _I8, _U8 = torch.bfloat16, torch.float32, torch.int32, torch.int8, torch.uint8


def _enqueue(name, index, *args):
    """The call with GPU `index` current and its current stream as last argument."""
    fn = getattr(_calls or step_lib(), name)
    if index == _device():
        st = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            st = fn(*args, _raw_stream(index))
    if st != 0:
        _check(name, st)


def _on(t, name, dtype, ndim, index):
    """_need(), and that t is on GPU `index`."""
    if (isinstance(t, torch.Tensor) and t.dtype is dtype and t.dim() == ndim and t.get_device() == index
            and t.is_contiguous()):
        return
    _need(t, name, dtype, ndim)
    raise ValueError(f"{name}: on {t.device}, expected cuda:{index}")


def _row_scales(rows, k, device):
    """Room for a scale per row; without columns the calls write none, and the
    scale of a row of nothing is that of a row of zeros."""
    return _empty((rows,), dtype=_F32, device=device) if k else torch.ones((rows,), dtype=_F32, device=device)


def _rmsnorm(name, x, weight, residual, eps, out_residual, code_dtype):
    eps = float(eps)
    module, at = _direct or _binding(x), _device()
    out = _done(name, module.rmsnorm(x, weight, residual, eps, out_residual, code_dtype is _I8, at, _raw_stream(at)))
    if out is not None:
        return out
    _need(x, "x", _BF16, 2)
    at = x.get_device()
    _on(weight, "weight", _BF16, 1, at)
    m, k = x.shape
    if weight.shape[0] != k:
        raise ValueError(f"weight has {weight.shape[0]} entries, x has {k} columns")
    h = x
    if residual is not None:
        _on(residual, "residual", _BF16, 2, at)
        if residual.shape != x.shape:
            raise ValueError(f"residual is {tuple(residual.shape)}, x is {tuple(x.shape)}")
        if out_residual is None:
            h = _empty_like(x)
        else:
            _on(out_residual, "out_residual", _BF16, 2, at)
            if out_residual.shape != x.shape:
                raise ValueError(f"out_residual is {tuple(out_residual.shape)}, x is {tuple(x.shape)}")
            h = out_residual
    elif out_residual is not None:
        raise ValueError("out_residual needs a residual")
    codes = _empty_like(x, dtype=code_dtype)
    if code_dtype is _U8:
        scales = _empty((m, k // 128), dtype=_F32, device=x.device)
    else:
        scales = _row_scales(m, k, x.device)
    if residual is None:
        _enqueue(name, at, m, k, x.data_ptr(), None, weight.data_ptr(), eps, None, codes.data_ptr(),
                 scales.data_ptr())
    else:
        _enqueue(name, at, m, k, x.data_ptr(), residual.data_ptr(), weight.data_ptr(), eps, h.data_ptr(),
                 codes.data_ptr(), scales.data_ptr())
    return codes, scales, h


def rmsnorm_quant(x, weight, residual=None, eps=1e-6, out_residual=None):
    """h = bf16(x + residual) (x without one); y = bf16(rmsnorm(h) * weight);
    returns (uint8 e4m3fn codes [M, K] and fp32 scales [M, K/128] of y,
    bitwise quant_act(y), and h). out_residual: where h is written
    (`residual` itself, for an update in place); allocated when None."""
    return _rmsnorm("fp8bq_rmsnorm_quant", x, weight, residual, eps, out_residual, _U8)


def rmsnorm_quant_i8(x, weight, residual=None, eps=1e-6, out_residual=None):
    """rmsnorm_quant() with int8 codes [M, K] and one fp32 scale per row [M],
    bitwise quant_act_i8(y)."""
    return _rmsnorm("fp8bq_rmsnorm_quant_i8", x, weight, residual, eps, out_residual, _I8)


def _quant_rows(name, x):
    rows, k = x.shape
    codes = _empty_like(x, dtype=_I8)
    scales = _row_scales(rows, k, x.device)
    _enqueue(name, x.get_device(), rows, k, x.data_ptr(), codes.data_ptr(), scales.data_ptr())
    return codes, scales


def quant_act_i8(a):
    """bf16 [M, K] -> (int8 codes [M, K], fp32 scales [M]), one scale per token."""
    _need(a, "a", torch.bfloat16, 2)
    return _quant_rows("fp8bq_quant_act_i8", a)


def quant_weight_i8(w):
    """fp32 [N, K] -> (int8 codes [N, K], fp32 scales [N]), one scale per output channel."""
    _need(w, "w", torch.float32, 2)
    return _quant_rows("fp8bq_quant_weight_i8", w)


def gemm_i8_workspace_bytes(m, n, k):
    """Device scratch bytes gemm_i8() can use on (M, N, K); raises on invalid sizes."""
    st = step_lib().fp8bq_gemm_i8_workspace_bytes(int(m), int(n), int(k))
    if st < 0:
        raise Fp8bqError("fp8bq_gemm_i8_workspace_bytes", st)
    return st


def _scratch(workspace, need, index):
    """(address, bytes) of a caller's uint8 workspace, or of one allocated
    here (None: `need` is 0), and the tensor that holds it."""
    if workspace is None:
        if need == 0:
            return None, 0, None
        workspace = _empty((need,), dtype=_U8, device=index)
    else:
        _on(workspace, "workspace", _U8, 1, index)
    return workspace.data_ptr(), workspace.shape[0], workspace


def gemm_i8(a_q, a_s, w_q, w_s, out=None, workspace=None):
    """C[m, n] = bf16(sum_k a_q[m, k] w_q[n, k] * (a_s[m] * w_s[n])): int8
    codes [M, K] and [N, K], fp32 scales [M] and [N], bf16 [M, N]. workspace
    (uint8, on the device): allocated when None and of use; one that is too
    small is not used. The result does not depend on it."""
    module, at = _direct or _binding(a_q), _device()
    done = _done("fp8bq_gemm_i8", module.gemm_i8(a_q, a_s, w_q, w_s, out, workspace, at, _raw_stream(at)))
    if done is not None:
        return done
    _need(a_q, "a_q", _I8, 2)
    at = a_q.get_device()
    _on(w_q, "w_q", _I8, 2, at)
    _on(a_s, "a_s", _F32, 1, at)
    _on(w_s, "w_s", _F32, 1, at)
    m, k = a_q.shape
    n, k2 = w_q.shape
    if k != k2:
        raise ValueError(f"K mismatch: a_q has {k}, w_q has {k2}")
    if a_s.shape[0] != m or w_s.shape[0] != n:
        raise ValueError(f"scale shapes {tuple(a_s.shape)}, {tuple(w_s.shape)} do not match M={m}, N={n}")
    if out is None:
        out = _empty((m, n), dtype=_BF16, device=a_q.device)
    else:
        _on(out, "out", _BF16, 2, at)
        if tuple(out.shape) != (m, n):
            raise ValueError(f"out must be [{m}, {n}]")
    scratch, nbytes, _keep = _scratch(workspace, gemm_i8_workspace_bytes(m, n, k) if workspace is None else 0, at)
    _enqueue("fp8bq_gemm_i8", at, m, n, k, a_q.data_ptr(), a_s.data_ptr(), w_q.data_ptr(), w_s.data_ptr(),
             out.data_ptr(), scratch, nbytes)
    return out


def verify_workspace_bytes(b, n_drafts, v):
    """Device scratch bytes verify_drafts() needs; raises on invalid sizes."""
    st = step_lib().fp8bq_verify_workspace_bytes(int(b), int(n_drafts), int(v))
    if st < 0:
        raise Fp8bqError("fp8bq_verify_workspace_bytes", st)
    return st


def verify_drafts(target_p, drafts, u_accept, u_sample, draft_p=None, draft_len=None, workspace=None):
    """Accept drafted tokens against the target's probabilities and draw the
    token after them.

    target_p [B, drafts + 1, V] and draft_p [B, drafts, V] (None: the drafts
    are certain) fp32 or bf16, drafts int32 [B, drafts], u_accept fp32 [B,
    drafts], u_sample fp32 [B], draft_len int32 [B] (None: all). Returns
    (tokens int32 [B, drafts + 1]: the accepted drafts, the drawn token, then
    -1; accepted int32 [B])."""
    module, at = _direct or _binding(target_p), _device()
    out = _done("fp8bq_verify_drafts", module.verify_drafts(target_p, drafts, u_accept, u_sample, draft_p, draft_len,
                                                            workspace, at, _raw_stream(at)))
    if out is not None:
        return out
    if not isinstance(target_p, torch.Tensor) or target_p.dtype not in (_F32, _BF16):
        raise TypeError("target_p: expected a float32 or bfloat16 torch.Tensor")
    kind = target_p.dtype
    _need(target_p, "target_p", kind, 3)
    at = target_p.get_device()
    _on(drafts, "drafts", _I32, 2, at)
    _on(u_accept, "u_accept", _F32, 2, at)
    _on(u_sample, "u_sample", _F32, 1, at)
    b, k = drafts.shape
    rows, places, v = target_p.shape
    if rows != b or places != k + 1:
        raise ValueError(f"target_p must be [{b}, {k + 1}, V], got {tuple(target_p.shape)}")
    if u_accept.shape != drafts.shape or u_sample.shape[0] != b:
        raise ValueError(f"u_accept must be [{b}, {k}] and u_sample [{b}]")
    q = lens = None
    if draft_p is not None:
        _on(draft_p, "draft_p", kind, 3, at)
        if tuple(draft_p.shape) != (b, k, v):
            raise ValueError(f"draft_p must be [{b}, {k}, {v}], got {tuple(draft_p.shape)}")
        q = draft_p.data_ptr() if k > 0 else None
    if draft_len is not None:
        _on(draft_len, "draft_len", _I32, 1, at)
        if draft_len.shape[0] != b:
            raise ValueError(f"draft_len must be [{b}]")
        lens = draft_len.data_ptr()
    scratch, nbytes, _keep = _scratch(workspace, verify_workspace_bytes(b, k, v) if workspace is None else 0, at)
    tokens = _empty((b, k + 1), dtype=_I32, device=target_p.device)
    accepted = _empty_like(u_sample, dtype=_I32)
    _enqueue("fp8bq_verify_drafts", at, b, k, v, F32 if kind is _F32 else BF16, target_p.data_ptr(), q,
             drafts.data_ptr(), lens, u_accept.data_ptr(), u_sample.data_ptr(), scratch, nbytes, tokens.data_ptr(),
             accepted.data_ptr())
    return tokens, accepted
