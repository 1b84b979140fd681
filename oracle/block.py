"""The block operators in float64 (numpy): block-scaled e4m3, the linear layer on
such operands, and the norms around a branch with gate and residual scale.

Written from the formulas of include/dcn_core.h; shares no code with the CUDA
library.  The quantiser is defined by fp32 operations (the scale, its reciprocal
and the scaled value are fp32 numbers), so its codes and scales are exact values,
not approximations; everything else is float64."""
from __future__ import annotations

import numpy as np

E4M3_MAX = 448.0
FLOOR = np.float32(7.0 * 2.0 ** -58)


def pitch(cols: int) -> int:
    return 16 * ((cols + 15) // 16)


def blocks(n: int) -> int:
    return (n + 127) // 128


def e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3
    fraction bits; exponent 0 is subnormal, 0x7F and 0xFF are NaN, no infinity."""
    code = np.arange(256)
    exp, frac = (code >> 3) & 15, code & 7
    mag = np.where(exp == 0, frac * 2.0 ** -9, (8 + frac) * 2.0 ** (exp - 10.0))
    mag = np.where((code & 127) == 127, np.nan, mag)
    return np.where(code >= 128, -mag, mag)


def e4m3_codes(v) -> np.ndarray:
    """Nearest code of each value (ties to the even code, clamped to +-448; NaN: 0x7F)."""
    v = np.asarray(v, dtype=np.float64)
    mags = e4m3_values()[:127]
    a = np.minimum(np.abs(np.nan_to_num(v)), E4M3_MAX)
    hi = np.minimum(np.searchsorted(mags, a), 126)  # first code not below a
    lo = np.maximum(hi - 1, 0)
    below, above = a - mags[lo], mags[hi] - a
    up = (above < below) | ((above == below) & (hi % 2 == 0))
    code = np.where(up, hi, lo) | np.where(np.signbit(v), 128, 0)
    return np.where(np.isnan(v), 127, code).astype(np.uint8)


def quantize(x, block_rows: int = 1):
    """(codes (rows, pitch(cols)) uint8, scales (blocks(cols), R) float32) of fp32 values x."""
    x = np.ascontiguousarray(x, dtype=np.float32)
    rows, cols = x.shape
    rb, kb = -(-rows // block_rows), blocks(cols)
    scales = np.empty((kb, rb), dtype=np.float32)
    codes = np.zeros((rows, pitch(cols)), dtype=np.uint8)
    for r in range(rb):
        for k in range(kb):
            rs, ks = slice(r * block_rows, min(rows, (r + 1) * block_rows)), slice(k * 128, min(cols, k * 128 + 128))
            v = x[rs, ks]
            if not np.isfinite(v).all():
                scales[k, r] = np.nan
                codes[rs, ks] = 127
                continue
            a = max(np.abs(v).max(), FLOOR)
            scales[k, r] = np.float32(a) / np.float32(448)
            codes[rs, ks] = e4m3_codes(v * (np.float32(448) / np.float32(a)))
    return codes, scales


def values(codes, scales, cols: int, block_rows: int = 1) -> np.ndarray:
    """What the codes stand for, float64 (rows, cols)."""
    v = e4m3_values()[np.asarray(codes)[:, :cols]]
    s = np.repeat(np.asarray(scales, dtype=np.float64), block_rows, axis=1)[:, :v.shape[0]]
    return v * np.repeat(s.T, 128, axis=1)[:, :cols]


def linear_fp8(a, a_scales, w, w_scales, K: int, bias=None):
    """(output, sum of the absolute terms), both float64 (M, Nout)."""
    av, wv = values(a, a_scales, K), values(w, w_scales, K, 128)
    out, mag = av @ wv.T, np.abs(av) @ np.abs(wv).T
    if bias is not None:
        out, mag = out + np.asarray(bias, np.float64), mag + np.abs(np.asarray(bias, np.float64))
    return out, mag


def _vec(p, n, dflt):
    return np.full(n, dflt) if p is None else np.asarray(p, dtype=np.float64)


def gate_rows(gate, rows_per_gate: int, M: int, C: int) -> np.ndarray:
    """The gate vector of every row, (M, C)."""
    if gate is None:
        return np.ones((M, C))
    g = np.asarray(gate, dtype=np.float64).reshape(-1, C)
    return g[np.arange(M) // rows_per_gate] if rows_per_gate > 0 else np.repeat(g, M, axis=0)


def stats(v, kind: str, eps: float):
    """(mean, 1 / deviation) of each row, (M, 1) each."""
    mean = v.mean(axis=1, keepdims=True) if kind == "layer" else np.zeros((v.shape[0], 1))
    return mean, 1.0 / np.sqrt(((v - mean) ** 2).mean(axis=1, keepdims=True) + eps)


def block_norm(x, y, gate=None, post_gamma=None, post_beta=None, pre_gamma=None, pre_beta=None, *,
               post="none", pre="layer", rows_per_gate=0, post_eps=1e-6, pre_eps=1e-6, alpha=1.0):
    """dict of r, h (with a pre norm) and the statistics, float64."""
    x = np.asarray(x, dtype=np.float64)
    M, C = x.shape
    out = {}
    r = alpha * x
    if y is not None:
        p = np.asarray(y, dtype=np.float64)
        if post != "none":
            mean, rstd = stats(p, post, post_eps)
            out["post_stats"] = np.concatenate([mean, rstd], axis=1).T
            p = (p - mean) * rstd * _vec(post_gamma, C, 1.0) + _vec(post_beta, C, 0.0)
        r = r + gate_rows(gate, rows_per_gate, M, C) * p
    out["r"] = r
    if pre != "none":
        mean, rstd = stats(r, pre, pre_eps)
        out["pre_stats"] = np.concatenate([mean, rstd], axis=1).T
        out["h"] = (r - mean) * rstd * _vec(pre_gamma, C, 1.0) + _vec(pre_beta, C, 0.0)
    return out


def _back(d, n, rstd, kind):
    g = d - n * (d * n).mean(axis=1, keepdims=True)
    if kind == "layer":
        g = g - d.mean(axis=1, keepdims=True)
    return rstd * g


def block_norm_backward(r, y, gate, post_gamma, post_beta, pre_gamma, post_stats, pre_stats,
                        grad_r, grad_h, *, post="none", pre="layer", rows_per_gate=0, alpha=1.0):
    """dict of the gradients: residual, branch, gate, post_gamma, post_beta,
    pre_gamma, pre_beta (float64), from the forward's r and statistics."""
    ref = next(v for v in (grad_r, grad_h) if v is not None)
    M, C = np.asarray(ref).shape
    out = {}
    dr = np.zeros((M, C)) if grad_r is None else np.asarray(grad_r, dtype=np.float64)
    if pre != "none":
        mean, rstd = (np.asarray(s, dtype=np.float64)[:, None] for s in pre_stats)
        m = (np.asarray(r, dtype=np.float64) - mean) * rstd
        dh = np.asarray(grad_h, dtype=np.float64)
        out["pre_gamma"], out["pre_beta"] = (dh * m).sum(axis=0), dh.sum(axis=0)
        dr = dr + _back(dh * _vec(pre_gamma, C, 1.0), m, rstd, pre)
    out["residual"] = alpha * dr
    if y is None:
        return out
    n, rstd = np.asarray(y, dtype=np.float64), np.ones((M, 1))
    if post != "none":
        mean, rstd = (np.asarray(s, dtype=np.float64)[:, None] for s in post_stats)
        n = (n - mean) * rstd
    g = gate_rows(gate, rows_per_gate, M, C)
    p = n * _vec(post_gamma, C, 1.0) + _vec(post_beta, C, 0.0)
    if gate is not None:
        count = -(-M // rows_per_gate) if rows_per_gate > 0 else 1
        out["gate"] = np.zeros((count, C))
        np.add.at(out["gate"], np.arange(M) // rows_per_gate if rows_per_gate > 0
                  else np.zeros(M, dtype=int), dr * p)
    dp = g * dr
    if post != "none":
        out["post_gamma"], out["post_beta"] = (dp * n).sum(axis=0), dp.sum(axis=0)
        out["branch"] = _back(dp * _vec(post_gamma, C, 1.0), n, rstd, post)
    else:
        out["branch"] = dp
    return out
