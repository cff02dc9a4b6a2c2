"""Row quantisation, the 8-bit product and the 8-bit expert FFN in float64, and
how far a correct fp32 / bf16 evaluation may be from them (tests only)."""
from __future__ import annotations

import numpy as np

BF16_HALF_STEP = 2.0 ** -8      # torch.finfo(bfloat16).eps / 2
F32_HALF_STEP = 2.0 ** -24


def bf16_round(a: np.ndarray) -> np.ndarray:
    """float64 -> nearest bf16 value (ties to even), as float64 (finite, normal values)."""
    m, e = np.frexp(a)
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


def quantize(x: np.ndarray):
    """(codes, scales) of the rows of x (float64): rne(127 x / max|x|), exact
    (the float64 quotient of an fp32 value is within 2^-52 of the true one,
    which is either n + 1/2 exactly or 2^-32 away from it)."""
    top = np.abs(x).max(-1, keepdims=True)
    with np.errstate(invalid="ignore", divide="ignore"):
        q = np.where(top > 0, np.rint(127.0 * x / np.where(top > 0, top, 1.0)), 0.0)
    return q, (top / 127.0)[..., 0]


def matmul(q, s, wq, ws, offsets=None):
    """The product over groups of rows; rows of no group are NaN."""
    out = np.full((q.shape[0], wq.shape[-2]), np.nan)
    ends = [0, q.shape[0]] if offsets is None else [int(v) for v in offsets]
    for g in range(len(ends) - 1):
        a, b = ends[g], ends[g + 1]
        out[a:b] = (q[a:b].astype(np.float64) @ wq[g].astype(np.float64).T) * s[a:b, None] * ws[g][None, :]
    return out


def silu(g):
    return g / (1.0 + np.exp(-g))


def expert_ffn(x: np.ndarray, w: dict, act: str):
    """One expert's rows: (y, bound).  ``w``: codes w1..w3 and scales s1..s3.

    ``bound`` is how far an fp32 evaluation that follows the definition may be
    from y before y's own rounding.  The intermediate's relative error is at
    most 2^-17 (three fp32 roundings a projection, and an exponential of
    |g| <= 20 good to 26 units of 2^-23), so its bf16 rounding can differ
    only for elements that close to a border, and by one bf16 step; such an
    element is at most 127 code steps and a bf16 step at most 2^-7 of it, so its
    code moves by at most one (two are allowed).  If the row's largest element
    is one of them, the row's scale moves by at most 2^-7 of itself and every
    code by at most one more.
    """
    q, s = quantize(x)
    gate = (q @ w["w1"].astype(np.float64).T) * s[:, None] * w["s1"][None, :]
    if act == "relu":
        h = np.maximum(gate, 0.0)
    else:
        assert np.abs(gate).max() <= 20.0
        h = silu(gate) * ((q @ w["w2"].astype(np.float64).T) * s[:, None] * w["s2"][None, :])
    hb = bf16_round(h)
    lo, hi = bf16_round(h * (1 - 2.0 ** -17)), bf16_round(h * (1 + 2.0 ** -17))
    risk = (lo != hb) | (hi != hb)
    hq, hs = quantize(hb)
    w3 = w["w3"].astype(np.float64) * w["s3"][:, None]
    y = (hq @ w3.T) * hs[:, None]
    top_risk = (risk & (np.abs(hb) >= np.abs(hb).max(-1, keepdims=True) * (1 - 2.0 ** -7))).any(-1)
    moved = np.where(top_risk[:, None], 1.0, 0.0) + 2.0 * risk
    bound = (moved @ np.abs(w3).T) * hs[:, None] + np.where(top_risk[:, None], 2.0 ** -7 * np.abs(y), 0.0)
    return y, bound + 4 * F32_HALF_STEP * np.abs(y)
