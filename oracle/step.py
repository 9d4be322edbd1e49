"""The operators around the linear layer (test infrastructure only): root-
mean-square norm with the residual's addition, int8 quantisation by rows, the
int8 product, and the verification of drafted tokens.

Page 3 (zskr.cn blog), section 3.3 fuses the norm with the quantisation and
section 2.2 uses INT8 weights; page 1 (SmartX blog), section "single-stream
optimisation", verifies k drafted tokens per step. The pages give no formulas;
the definitions are the ones written out in include/fp8bq_step.h.

* norm: h = bf16(x + r) with the sum in fp32; mean square, root and reciprocal
  in fp64, rounded once to fp32 (held to the largest finite number); y =
  bf16((h * inv) * w) in fp32.
* int8 rows: scale = amax / 127 in fp32 (1 where that is 0), code =
  rint(x / scale) held to -127 .. 127.
* product: the integer sums in fp64 (exact below 2^53), rounded to fp32, times
  the fp32 product of the two scales, rounded to bf16.
* verification: comparisons and sums in Python's whole numbers and Fractions.
"""

from fractions import Fraction

import numpy as np

from .quant import _as_float32

F32 = np.float32


def bf16_round(x) -> np.ndarray:
    """fp32 -> nearest bf16 (ties to even), as fp32. NaN stays NaN."""
    b = np.ascontiguousarray(x, dtype=F32).view(np.uint32).astype(np.uint64)
    r = ((b + 0x7FFF + ((b >> 16) & 1)) & 0xFFFF0000).astype(np.uint32)
    out = r.view(F32).reshape(np.shape(x))
    return np.where(np.isnan(x), np.asarray(x, F32), out)


def rmsnorm_ref(x, w, r=None, eps=1e-6):
    """x, r [M, K], w [K] holding bf16 values. Returns (y, h) as float32
    holding bf16 values."""
    x, w = _as_float32(x), _as_float32(w)
    h = x if r is None else bf16_round(x + _as_float32(r))
    mean = (h.astype(np.float64) ** 2).sum(axis=1, keepdims=True) / x.shape[1]
    inv = np.minimum(1.0 / np.sqrt(mean + eps), np.finfo(F32).max).astype(F32)
    return bf16_round((h * inv) * w), h


def quant_rows_i8_ref(x):
    """x [M, K] -> (int8 codes [M, K], float32 scales [M])."""
    x = _as_float32(x)
    amax = np.abs(x).max(axis=1).astype(F32)
    s = np.divide(amax, F32(127.0), dtype=F32)
    s = np.where(s > 0, s, F32(1.0)).astype(F32)
    q = np.clip(np.divide(x, s[:, None], dtype=F32), F32(-127.0), F32(127.0))
    return np.rint(q).astype(np.int8), s


def gemm_i8_ref(a_q, a_s, w_q, w_s):
    """Returns the bf16 results as float32."""
    sums = a_q.astype(np.float64) @ w_q.astype(np.float64).T
    scales = (np.asarray(a_s, F32)[:, None] * np.asarray(w_s, F32)[None, :]).astype(F32)
    return bf16_round(sums.astype(F32) * scales)


def weight_units(w) -> np.ndarray:
    """fp32 weights -> whole numbers of 2^-32 (ties to even; 0 for NaN and
    below, at most 2^32 - 1), int64."""
    w = np.asarray(w, dtype=F32).astype(np.float64)
    w = np.where(np.isnan(w), 0.0, w)
    return np.clip(np.rint(w * 2.0 ** 32), 0, 2 ** 32 - 1).astype(np.int64)


def draw_ref(units, u) -> int:
    """Lowest index whose running sum exceeds floor(S z / 2^32), z =
    floor(u 2^32); -1 where S is 0."""
    total = int(units.sum())
    if total == 0:
        return -1
    z = min(int(Fraction(float(u)) * 2 ** 32), 2 ** 32 - 1)
    goal = total * z // 2 ** 32
    return int(np.searchsorted(np.cumsum(units), goal, side="right"))


def verify_ref(target, drafts, u_accept, u_sample, draft=None, draft_len=None):
    """target [B, k + 1, V], draft [B, k, V] or None, drafts [B, k] (numpy).
    Returns (tokens int64 [B, k + 1], accepted int64 [B])."""
    b, k = drafts.shape
    v = target.shape[2]
    tokens = np.full((b, k + 1), -1, dtype=np.int64)
    accepted = np.zeros(b, dtype=np.int64)
    for i in range(b):
        n = k if draft_len is None else min(max(int(draft_len[i]), 0), k)
        r = 0
        while r < n:
            d = int(drafts[i, r])
            if not 0 <= d < v:
                break
            p = float(target[i, r, d])
            q = 1.0 if draft is None else float(draft[i, r, d])
            u = float(u_accept[i, r])
            if not (np.isfinite([u, p, q]).all() and Fraction(u) * Fraction(q) < Fraction(p)):
                break
            tokens[i, r] = d
            r += 1
        row = np.asarray(target[i, r], dtype=F32)
        units = weight_units(row)
        if r < n:
            away = np.zeros(v, dtype=F32)
            if draft is not None:
                away = np.asarray(draft[i, r], dtype=F32)
            elif 0 <= int(drafts[i, r]) < v:
                away[int(drafts[i, r])] = 1.0
            with np.errstate(invalid="ignore"):
                left = weight_units((row - away).astype(F32))
            if left.sum() > 0:
                units = left
        tokens[i, r] = draw_ref(units, u_sample[i])
        accepted[i] = r
    return tokens, accepted
