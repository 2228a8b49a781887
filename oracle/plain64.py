"""Plain float64 forms of the int8 sub-layer's operators, in numpy.

TEST INFRASTRUCTURE ONLY, as oracle.py: no code, constant or layout is shared
with the CUDA path. Inputs are float64 arrays (bf16 values widened exactly) or
integer codes; every function is the operator's definition, written request
by request.
"""

from __future__ import annotations

import numpy as np

NORM_RMS, NORM_LAYER, NORM_NONE = 0, 1, 2


def _requests(cu):
    return [(s, int(cu[s]), int(cu[s + 1])) for s in range(len(cu) - 1)]


def norm_modulate(x, *, branch=None, gate_res=None, weight=None, shift=None, scale=None, cu_seqlens=None,
                  norm_type=NORM_RMS, eps=1e-6):
    """Returns (x', h): the residual stream and the row that is coded."""
    x = np.array(x, dtype=np.float64)
    cu = np.array([0, x.shape[0]]) if cu_seqlens is None else np.asarray(cu_seqlens)
    if branch is not None:
        for s, a, b in _requests(cu):
            x[a:b] += branch[a:b] if gate_res is None else np.asarray(gate_res[s], np.float64) * branch[a:b]
    h = x.copy()
    if norm_type == NORM_LAYER:
        h -= h.mean(axis=1, keepdims=True)
    if norm_type != NORM_NONE:
        h /= np.sqrt((h * h).mean(axis=1, keepdims=True) + eps)
    if weight is not None:
        h *= weight
    if scale is not None:
        for s, a, b in _requests(cu):
            h[a:b] = h[a:b] * (1.0 + np.asarray(scale[s], np.float64)) + np.asarray(shift[s], np.float64)
    return x, h


def row_scales(h):
    """max |h| / 127 of each row, 1 where the row is zero."""
    amax = np.abs(h).max(axis=1)
    return np.where(amax == 0.0, 1.0, amax / 127.0)


def quantize_rows(h):
    """(codes int8, scales): h / scale to the nearest integer, ties to even."""
    s = row_scales(h)
    return np.rint(h / s[:, None]).astype(np.int8), s


def linear_i8(a8, a_scale, w8, w_scale):
    """a_scale[t] w_scale[n] sum_k a8[t, k] w8[n, k]; the sums are exact (whole
    numbers below 2^53 in float64)."""
    sums = a8.astype(np.float64) @ w8.astype(np.float64).T
    return sums * np.asarray(a_scale, np.float64)[:, None] * np.asarray(w_scale, np.float64)[None, :]


def gated_residual(y, x, gate_res, cu_seqlens):
    out = np.array(x, dtype=np.float64)
    for s, a, b in _requests(cu_seqlens):
        out[a:b] += np.asarray(gate_res[s], np.float64) * y[a:b]
    return out


def swiglu(y):
    F = y.shape[1] // 2
    g, u = y[:, :F], y[:, F:]
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g)) * u


def cross_attention(q, k, v, cu_q, cu_k, scale):
    """q [Tq, H, D], k and v [Tk, Hkv, D]. Returns (o, lse [H, Tq], spread):
    spread is the softmax-weighted mean of |v|, by which a relative error of
    the probabilities moves o. Rows of no request are 0 (lse -inf)."""
    Tq, H, D = q.shape
    group = H // k.shape[1]
    o, spread = np.zeros((Tq, H, D)), np.zeros((Tq, H, D))
    lse = np.full((H, Tq), -np.inf)
    for (_, qa, qb), (_, ka, kb) in zip(_requests(cu_q), _requests(cu_k)):
        if qa == qb or ka == kb:
            continue
        for h in range(H):
            s = scale * (q[qa:qb, h] @ k[ka:kb, h // group].T)
            top = s.max(axis=1, keepdims=True)
            p = np.exp(s - top)
            z = p.sum(axis=1, keepdims=True)
            o[qa:qb, h] = (p / z) @ v[ka:kb, h // group]
            spread[qa:qb, h] = (p / z) @ np.abs(v[ka:kb, h // group])
            lse[h, qa:qb] = (top + np.log(z))[:, 0]
    return o, lse, spread
