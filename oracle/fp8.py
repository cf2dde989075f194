"""Float64 numpy oracle of the experts on E4M3 codes with block scales.

TEST INFRASTRUCTURE, from the definitions (OCP 8-bit Floating Point
Specification, E4M3: 4 exponent bits with bias 7, 3 fraction bits, the code
with all bits set is NaN, no infinity), sharing no code with the CUDA path.
"""
from __future__ import annotations

import numpy as np


def e4m3(code: int) -> float:
    sign = -1.0 if code & 0x80 else 1.0
    e, f = (code >> 3) & 15, code & 7
    if e == 15 and f == 7:
        return float("nan")
    return sign * (f / 8 * 2.0 ** -6 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7))


VALUES = np.array([e4m3(c) for c in range(256)])
_POS = VALUES[:127]                        # ascending, 0 to 448


def encode(v):
    """Codes of v by nearest value, ties to the even code, magnitudes past 448
    saturated; NaN and infinities to the NaN code."""
    v = np.asarray(v, dtype=np.float64)
    a = np.minimum(np.abs(np.nan_to_num(v, nan=0.0, posinf=0.0, neginf=0.0)), 448.0)
    hi = np.searchsorted(_POS, a, side="left").clip(0, 126)
    lo = (hi - 1).clip(0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code |= np.where(np.signbit(v), 0x80, 0).astype(np.uint8)
    return np.where(np.isfinite(v), code, np.uint8(0x7F))


def quantize_weights(w):
    """float32 w [R, C] -> (codes, float32 scales) per 128 x 128 block."""
    w = np.asarray(w, dtype=np.float32)
    R, C = w.shape
    q = np.zeros((R, C), dtype=np.uint8)
    s = np.ones((-(-R // 128), -(-C // 128)), dtype=np.float32)
    for i in range(s.shape[0]):
        for j in range(s.shape[1]):
            b = w[128 * i:128 * i + 128, 128 * j:128 * j + 128]
            amax = np.abs(b[np.isfinite(b)]).max(initial=np.float32(0))
            if amax > 0:
                s[i, j] = max(np.float32(amax) / np.float32(448), np.float32(2.0 ** -126))
            with np.errstate(invalid="ignore"):
                q[128 * i:128 * i + 128, 128 * j:128 * j + 128] = encode(b / s[i, j])
    return q, s


def dequantize(q, s):
    w = VALUES[np.asarray(q)]
    s = np.asarray(s, dtype=np.float64)
    R, C = w.shape
    return w * np.repeat(np.repeat(s, 128, 0)[:R], 128, 1)[:, :C]


def round_rows(v):
    """v rounded to codes times the smallest power of two per row and 128
    columns that keeps the block within 448 (at least 2^-126)."""
    v = np.asarray(v, dtype=np.float64)
    out = np.empty_like(v)
    for c in range(0, v.shape[1], 128):
        b = v[:, c:c + 128]
        top = np.abs(np.where(np.isfinite(b), b, 0)).max(axis=1, keepdims=True)
        e = np.zeros(top.shape)
        for i, a in np.ndenumerate(top):
            k = -126
            if a > 448 * 2.0 ** -126:
                m, k = np.frexp(a)
                k = int(k) - 9 + (1 if m > 0.875 else 0)       # 448 = 0.875 * 2^9
                k = max(k, -126)
            e[i] = 2.0 ** k
        out[:, c:c + 128] = VALUES[encode(b / e)] * e
    return out


def expert(x, gu_q, gu_s, dn_q, dn_s):
    """x [n, H] through one gated expert; gu_s [2, ...]: gate and up scales."""
    I = gu_q.shape[0] // 2
    xr = round_rows(x)
    with np.errstate(invalid="ignore", over="ignore"):
        g = xr @ dequantize(gu_q[:I], gu_s[0]).T
        u = xr @ dequantize(gu_q[I:], gu_s[1]).T
        return round_rows(g / (1 + np.exp(-g)) * u) @ dequantize(dn_q, dn_s).T


def slots(x, perm, offsets, topk_w, fp8, k, routed_scale=1.0):
    """y_slots [T*k + S*T, H] given the plan; fp8: the expert set's arrays."""
    x = np.asarray(x, dtype=np.float64)
    T, H = x.shape
    S = 0 if fp8.get("sh_down_q") is None else fp8["sh_down_q"].shape[0]
    y = np.zeros((T * (k + S), H))
    w = np.asarray(topk_w, dtype=np.float64).reshape(-1)
    for e in range(len(offsets) - 1):
        a, b = int(offsets[e]), int(offsets[e + 1])
        if a == b:
            continue
        p = np.asarray(perm[a:b])
        y[a:b] = expert(x[p // k], fp8["gate_up_q"][e], fp8["gate_up_s"][e], fp8["down_q"][e],
                        fp8["down_s"][e]) * (routed_scale * w[p])[:, None]
    for s in range(S):
        y[T * k + s * T:T * k + (s + 1) * T] = expert(
            x, fp8["sh_gate_up_q"][s], fp8["sh_gate_up_s"][s], fp8["sh_down_q"][s],
            fp8["sh_down_s"][s])
    return y
