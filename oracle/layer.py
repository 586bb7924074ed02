"""fp64 forms of the operators around a recurrent layer, written from their definitions (numpy, no code
shared with the library).  Each returns, next to its result, the sum of the magnitudes of the terms
behind every value, which the tests' error bounds are multiples of."""
from __future__ import annotations

import numpy as np

BLOCK = 128
FP8_MAX = 448.0
AMAX_FLOOR = 1e-30


def rmsnorm_blocks(x, residual, weight, eps):
    """(z, y / scale, scale): the sum, the values to be rounded to e4m3 and the scale of each 128 of them."""
    z = np.asarray(x, np.float64) if residual is None else np.asarray(x, np.float64) + np.asarray(residual, np.float64)
    y = z / np.sqrt((z * z).mean(1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    D = z.shape[1]
    scale = np.empty((z.shape[0], -(-D // BLOCK)))
    ratio = np.empty_like(y)
    for i, c in enumerate(range(0, D, BLOCK)):
        part = y[:, c:c + BLOCK]
        scale[:, i] = np.maximum(np.abs(part).max(1), AMAX_FLOOR) / FP8_MAX
        ratio[:, c:c + BLOCK] = part / scale[:, i:i + 1]
    return z, ratio, scale


def block_matmul(a, a_scale, b, b_scale):
    """(out, sum of |terms|) of the product of block-scaled rows; a, b hold the e4m3 values."""
    a, b = np.asarray(a, np.float64), np.asarray(b, np.float64)
    K, N = a.shape[1], b.shape[0]
    kb = np.arange(K) // BLOCK
    nb = np.arange(N) // BLOCK
    wa = a * np.asarray(a_scale, np.float64)[:, kb]
    wb = b * np.asarray(b_scale, np.float64)[nb][:, kb]
    return wa @ wb.T, np.abs(wa) @ np.abs(wb).T


def linear_recurrence(q, k, v, g, h0=None, cu=None, scale=1.0):
    """Token by token.  q, k: [T, H, dk]; v: [T, H, dv]; g: [T, H] or [H]; h0: [B, H, dk, dv]; cu: [B + 1].
    Returns (out, final states, sum of |terms| of out, of the states)."""
    q, k, v = (np.asarray(t, np.float64) for t in (q, k, v))
    T, H, dk = q.shape
    dv = v.shape[2]
    g = np.asarray(g, np.float64)
    e = np.broadcast_to(np.exp(g), (T, H))
    cu = [0, T] if cu is None else [int(c) for c in cu]
    B = len(cu) - 1
    S = np.zeros((B, H, dk, dv)) if h0 is None else np.array(h0, np.float64)
    M = np.abs(S)
    out, mag = np.zeros((T, H, dv)), np.zeros((T, H, dv))
    for b in range(B):
        for t in range(cu[b], cu[b + 1]):
            S[b] = e[t][:, None, None] * S[b] + k[t][:, :, None] * v[t][:, None, :]
            M[b] = e[t][:, None, None] * M[b] + np.abs(k[t])[:, :, None] * np.abs(v[t])[:, None, :]
            out[t] = scale * np.einsum("hkv,hk->hv", S[b], q[t])
            mag[t] = abs(scale) * np.einsum("hkv,hk->hv", M[b], np.abs(q[t]))
    return out, S, mag, M
