"""fp64 oracle of the operators of an attention layer over a paged cache: the step's bookkeeping as a list of
blocks, rotary positions as complex numbers, and attention row by row over the keys that a row sees."""
from __future__ import annotations

import numpy as np


def block_tables(counts, lengths, tables, free, block_size, max_tokens, num_blocks):
    """One step on Python lists.  free: the free blocks in order.  Returns (slots, positions, offsets, new lengths, tables,
    free) with the blocks given back at the end of `free`, or None where the step does nothing."""
    tables, free = [list(t) for t in tables], list(free)
    blocks = lambda n: -(-n // block_size)  # noqa: E731
    width = len(tables[0]) if tables else 0
    new = [a + c for a, c in zip(lengths, counts)]
    if any(not 0 <= a <= width * block_size for a in list(lengths) + new) or sum(max(c, 0) for c in counts) > max_tokens:
        return None
    given, taken = [], 0
    for n, (a, b) in enumerate(zip(lengths, new)):
        given += tables[n][blocks(b):blocks(a)]
        taken += max(0, blocks(b) - blocks(a))
    if taken > len(free):
        return None
    slots, positions, offsets = [], [], [0]
    for n, (a, b) in enumerate(zip(lengths, new)):
        for i in range(blocks(a), blocks(b)):
            tables[n][i] = free.pop(0)
        for p in range(a, b):
            slots.append(tables[n][p // block_size] * block_size + p % block_size)
            positions.append(p)
        offsets.append(len(slots))
    pad = max_tokens - len(slots)
    return slots + [-1] * pad, positions + [0] * pad, offsets, new, tables, free + given


def rotate(x, positions, inv_freq, axis, interleaved):
    """x: [T, heads, d]; positions: [axes, T].  Each pair as a complex number times e^{i angle}."""
    x = np.array(x, np.float64)
    n = len(inv_freq)
    angle = np.stack([positions[a].astype(np.longdouble) * np.longdouble(f) for a, f in zip(axis, inv_freq)], 1) if n else \
        np.zeros((len(x), 0), np.longdouble)
    unit = (np.cos(angle) + 1j * np.sin(angle)).astype(np.complex128)[:, None]
    a, b = (x[..., 0:2 * n:2], x[..., 1:2 * n:2]) if interleaved else (x[..., :n], x[..., n:2 * n])
    z = (a + 1j * b) * unit
    y = x.copy()
    if interleaved:
        y[..., 0:2 * n:2], y[..., 1:2 * n:2] = z.real, z.imag
    else:
        y[..., :n], y[..., n:2 * n] = z.real, z.imag
    return y


def visible(length, tokens, window, sinks, masks=None):
    """[tokens, length] truth values: which keys each of a request's last tokens sees.  masks: for each drafted token
    the set of drafted tokens it sees, or None (causal)."""
    before, j = length - tokens, np.arange(length)
    rows = []
    for i in range(tokens):
        p = before + i if masks is None else before + len(masks[i]) - 1
        see = (j <= p) if masks is None else (j < before)
        if window > 0:
            see = see & ((j > p - window) | (j < sinks))
        if masks is not None:
            see = see | np.isin(j - before, sorted(masks[i]))
        rows.append(see)
    return np.array(rows, bool).reshape(tokens, length)


def attention(q, k, v, see, scale):
    """q: [n, H, d]; k, v: [length, Hkv, d]; see: [n, length].  Returns (out, sum of p |v|, largest sum |q||k| scale of a
    row's keys), the last two being what error bounds need.  A row that sees nothing is zero."""
    n, H, d = q.shape
    G = H // k.shape[1]
    out, mag, size = np.zeros((n, H, d)), np.zeros((n, H, d)), np.zeros((n, H, 1))
    keep = see.any(0)
    k, v, see = k[keep], v[keep], see[:, keep]
    some = see.any(1)
    if not some.any():
        return out, mag, size
    for h in range(H):
        kh, vh = k[:, h // G], v[:, h // G]
        s = np.where(see, scale * (q[:, h] @ kh.T), -np.inf)
        top = np.where(some, s.max(1), 0.0)
        p = np.exp(s - top[:, None])
        p /= np.where(some, p.sum(1), 1.0)[:, None]
        out[:, h], mag[:, h] = p @ vh, p @ np.abs(vh)
        size[:, h, 0] = np.where(see, scale * (np.abs(q[:, h]) @ np.abs(kh).T), 0).max(1)
    return out, mag, size
