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
tensors' device.
"""

import ctypes

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


def _enqueue(name, device, *args):
    """The call with `device` current and its current stream as last argument."""
    fn = getattr(step_lib(), name)
    if device.index == torch.cuda.current_device():
        st = fn(*args, torch.cuda.current_stream().cuda_stream)
    else:
        with torch.cuda.device(device):
            st = fn(*args, torch.cuda.current_stream().cuda_stream)
    _check(name, st)


def _same_device(device, **tensors):
    for name, t in tensors.items():
        if t is not None and t.device != device:
            raise ValueError(f"{name}: on {t.device}, expected {device}")


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rmsnorm(name, x, weight, residual, eps, out_residual, scale_cols, code_dtype):
    _need(x, "x", torch.bfloat16, 2)
    _need(weight, "weight", torch.bfloat16, 1)
    m, k = x.shape
    if weight.shape[0] != k:
        raise ValueError(f"weight has {weight.shape[0]} entries, x has {k} columns")
    h = None
    if residual is not None:
        _need(residual, "residual", torch.bfloat16, 2)
        if residual.shape != x.shape:
            raise ValueError(f"residual is {tuple(residual.shape)}, x is {tuple(x.shape)}")
        if out_residual is None:
            h = torch.empty_like(x)
        else:
            _need(out_residual, "out_residual", torch.bfloat16, 2)
            if out_residual.shape != x.shape:
                raise ValueError(f"out_residual is {tuple(out_residual.shape)}, x is {tuple(x.shape)}")
            h = out_residual
    elif out_residual is not None:
        raise ValueError("out_residual needs a residual")
    _same_device(x.device, weight=weight, residual=residual, out_residual=h)
    codes = torch.empty((m, k), dtype=code_dtype, device=x.device)
    scales = torch.empty((m, scale_cols(k)) if scale_cols else (m,), dtype=torch.float32, device=x.device)
    _enqueue(name, x.device, m, k, _ptr(x), _ptr(residual), _ptr(weight), float(eps), _ptr(h), _ptr(codes),
             _ptr(scales))
    return codes, scales, x if h is None else h


def _groups(k):
    return k // 128 if k % 128 == 0 else 0


def rmsnorm_quant(x, weight, residual=None, eps=1e-6, out_residual=None):
    """h = bf16(x + residual) (x without one); y = bf16(rmsnorm(h) * weight);
    returns (uint8 e4m3fn codes [M, K] and fp32 scales [M, K/128] of y,
    bitwise quant_act(y), and h). out_residual: where h is written
    (`residual` itself, for an update in place); allocated when None."""
    return _rmsnorm("fp8bq_rmsnorm_quant", x, weight, residual, eps, out_residual, _groups, torch.uint8)


def rmsnorm_quant_i8(x, weight, residual=None, eps=1e-6, out_residual=None):
    """rmsnorm_quant() with int8 codes [M, K] and one fp32 scale per row [M],
    bitwise quant_act_i8(y)."""
    return _rmsnorm("fp8bq_rmsnorm_quant_i8", x, weight, residual, eps, out_residual, None, torch.int8)


def _quant_rows(name, x):
    rows, k = x.shape
    codes = torch.empty((rows, k), dtype=torch.int8, device=x.device)
    scales = torch.empty((rows,), dtype=torch.float32, device=x.device)
    _enqueue(name, x.device, rows, k, _ptr(x), _ptr(codes), _ptr(scales))
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


def _scratch(workspace, need, device):
    """A caller's uint8 workspace, or one allocated here; None where none is needed."""
    if workspace is None:
        return torch.empty(need, dtype=torch.uint8, device=device) if need > 0 else None
    _need(workspace, "workspace", torch.uint8, 1)
    _same_device(device, workspace=workspace)
    return workspace


def gemm_i8(a_q, a_s, w_q, w_s, out=None, workspace=None):
    """C[m, n] = bf16(sum_k a_q[m, k] w_q[n, k] * (a_s[m] * w_s[n])): int8
    codes [M, K] and [N, K], fp32 scales [M] and [N], bf16 [M, N]. workspace
    (uint8, on the device): allocated when None and of use; one that is too
    small is not used. The result does not depend on it."""
    _need(a_q, "a_q", torch.int8, 2)
    _need(w_q, "w_q", torch.int8, 2)
    _need(a_s, "a_s", torch.float32, 1)
    _need(w_s, "w_s", torch.float32, 1)
    m, k = a_q.shape
    n, k2 = w_q.shape
    if k != k2:
        raise ValueError(f"K mismatch: a_q has {k}, w_q has {k2}")
    if a_s.shape[0] != m or w_s.shape[0] != n:
        raise ValueError(f"scale shapes {tuple(a_s.shape)}, {tuple(w_s.shape)} do not match M={m}, N={n}")
    device = a_q.device
    if out is None:
        out = torch.empty((m, n), dtype=torch.bfloat16, device=device)
    else:
        _need(out, "out", torch.bfloat16, 2)
        if tuple(out.shape) != (m, n):
            raise ValueError(f"out must be [{m}, {n}]")
    _same_device(device, w_q=w_q, a_s=a_s, w_s=w_s, out=out)
    workspace = _scratch(workspace, gemm_i8_workspace_bytes(m, n, k) if workspace is None else 0, device)
    _enqueue("fp8bq_gemm_i8", device, m, n, k, _ptr(a_q), _ptr(a_s), _ptr(w_q), _ptr(w_s), _ptr(out),
             _ptr(workspace), 0 if workspace is None else workspace.numel())
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
    if not isinstance(target_p, torch.Tensor) or target_p.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError("target_p: expected a float32 or bfloat16 torch.Tensor")
    _need(target_p, "target_p", target_p.dtype, 3)
    _need(drafts, "drafts", torch.int32, 2)
    _need(u_accept, "u_accept", torch.float32, 2)
    _need(u_sample, "u_sample", torch.float32, 1)
    b, k = drafts.shape
    v = target_p.shape[2]
    if tuple(target_p.shape[:2]) != (b, k + 1):
        raise ValueError(f"target_p must be [{b}, {k + 1}, V], got {tuple(target_p.shape)}")
    if tuple(u_accept.shape) != (b, k) or u_sample.shape[0] != b:
        raise ValueError(f"u_accept must be [{b}, {k}] and u_sample [{b}]")
    if draft_p is not None:
        _need(draft_p, "draft_p", target_p.dtype, 3)
        if tuple(draft_p.shape) != (b, k, v):
            raise ValueError(f"draft_p must be [{b}, {k}, {v}], got {tuple(draft_p.shape)}")
        if k == 0:
            draft_p = None
    if draft_len is not None:
        _need(draft_len, "draft_len", torch.int32, 1)
        if draft_len.shape[0] != b:
            raise ValueError(f"draft_len must be [{b}]")
    device = target_p.device
    _same_device(device, drafts=drafts, u_accept=u_accept, u_sample=u_sample, draft_p=draft_p, draft_len=draft_len)
    need = verify_workspace_bytes(b, k, v)
    workspace = _scratch(workspace, need, device)
    tokens = torch.empty((b, k + 1), dtype=torch.int32, device=device)
    accepted = torch.empty((b,), dtype=torch.int32, device=device)
    _enqueue("fp8bq_verify_drafts", device, b, k, v, F32 if target_p.dtype == torch.float32 else BF16, _ptr(target_p),
             _ptr(draft_p), _ptr(drafts), _ptr(draft_len), _ptr(u_accept), _ptr(u_sample), _ptr(workspace),
             0 if workspace is None else workspace.numel(), _ptr(tokens), _ptr(accepted))
    return tokens, accepted
