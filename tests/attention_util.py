"""Inputs, checks and error bounds for the tests of the attention layer's operators."""
from __future__ import annotations

import numpy as np
import torch

import gated_delta_rule_08_gb300 as kda
from layer_util import F32, HALF, f64, gen, randn, within
from oracle import attention as oracle

BF = torch.bfloat16


def ints(values, device="cuda"):
    return torch.tensor(values, dtype=torch.int32, device=device)


def tree_masks(n, seed, children=3):
    """For each of n drafted tokens the set of those it sees: a random tree's ancestors and itself."""
    r = np.random.default_rng(seed)
    seen = []
    for j in range(n):
        parent = j - 1 - int(r.integers(0, children))
        seen.append((seen[parent] if parent >= 0 else set()) | {j})
    return seen


def mask_words(masks, words):
    """The sets of all drafted tokens as int64 [T, words]."""
    out = np.zeros((len(masks), words), np.uint64)
    for i, m in enumerate(masks):
        for j in m:
            out[i, j // 64] |= np.uint64(1 << (j % 64))
    return torch.from_numpy(out.view(np.int64))


class Batch:
    """Requests with `cached` tokens and `new` ones in a paged cache.  What no new token sees holds NaN: tokens behind a
    request's last, blocks of nobody, and (window) keys before the window; table entries of blocks that are wholly so
    are -1."""

    def __init__(self, cached, new, H=8, Hkv=2, d=128, block=16, window=0, sinks=0, seed=0, masks=None, layout="token",
                 poison=True, spare=3, packed=False, scale=None):
        r = gen(seed)
        self.cached, self.new, self.H, self.Hkv, self.d, self.block = list(cached), list(new), H, Hkv, d, block
        self.window, self.sinks, self.masks = window, sinks, masks
        self.scale = d ** -0.5 if scale is None else scale
        lengths = [a + b for a, b in zip(cached, new)]
        held = [-(-n // block) for n in lengths]
        blocks, width = sum(held) + spare, max(held + [1]) + 1
        order = np.random.default_rng(seed).permutation(blocks)
        T = sum(new)
        row = randn(r, T, H * d + (24 if packed else 0), dtype=BF)
        self.q = row[:, :H * d].view(T, H, d)
        shape = (blocks, Hkv, block, d) if layout == "head" else (blocks, block, Hkv, d)
        self.k, self.v = (torch.full(shape, float("nan") if poison else 0.0, dtype=BF, device="cuda") for _ in range(2))
        if layout == "head":
            self.k, self.v = self.k.transpose(1, 2), self.v.transpose(1, 2)
        table = np.full((len(new), width), -1, np.int32)
        self.keys, self.values, self.see = [], [], []
        at = 0
        for n, (a, b) in enumerate(zip(cached, new)):
            length, mine = a + b, order[at:at + held[n]]
            at += held[n]
            see = oracle.visible(length, b, window, sinks, None if masks is None else masks[n]) if b else np.zeros((0, length), bool)
            k, v = randn(r, length, Hkv, d, dtype=BF), randn(r, length, Hkv, d, dtype=BF)
            # every drafted and new token is there; of the cached ones, those that somebody sees
            there = torch.from_numpy(np.concatenate([see[:, :a].any(0), np.ones(b, bool)])).cuda()
            slot = torch.from_numpy(mine.repeat(block)[:length] * block + np.arange(length) % block).cuda()
            fill = there if poison else torch.ones_like(there)
            self.k[slot[fill] // block, slot[fill] % block] = k[fill]
            self.v[slot[fill] // block, slot[fill] % block] = v[fill]
            for i in range(held[n]):
                if not poison or bool(there[i * block:(i + 1) * block].any()):
                    table[n, i] = mine[i]
            self.keys.append(f64(k))
            self.values.append(f64(v))
            self.see.append(see)
        self.table = torch.from_numpy(table).cuda()
        self.lengths = ints(lengths)
        self.cu = ints(np.concatenate([[0], np.cumsum(new)]).astype(int).tolist())

    def options(self):
        return dict(window=self.window, sinks=self.sinks, scale=self.scale)

    def run(self, q=None, **kw):
        args = (self.q if q is None else q, self.k, self.v, self.table, self.lengths)
        kw = {**self.options(), **kw}
        if self.masks is not None:
            words = max(1, -(-max(self.new + [1]) // 64))
            mask = mask_words([m for ms in self.masks for m in ms], words).cuda()
            return kda.kda_tree_attention(*args, self.cu, mask, **kw)
        return kda.kda_window_attention_fwd(*args, self.cu, **kw)

    def step(self, **kw):
        return kda.kda_window_attention_decode_step(self.q, self.k, self.v, self.table, self.lengths, **{**self.options(), **kw})

    def check(self, out, what=""):
        """Scores are sums of d products in fp32 (each step F32 of the magnitudes, and as much again for scaling and the
        reference), exponentials and sums over n weights likewise, each weight is rounded to bf16 once before its product
        with the values (HALF), and the result once more."""
        assert kda.kda_get_device_error() == 0
        half, t = HALF[BF], 0
        for n, b in enumerate(self.new):
            want, mag, size = oracle.attention(f64(self.q[t:t + b]), self.keys[n], self.values[n], self.see[n], self.scale)
            inner = (half + 4 * F32 * (2 * (self.d + 4) * size + len(self.keys[n]) + 16)) * mag
            within(out[t:t + b], want, half * (np.abs(want) + inner) + inner, (what, "request", n))
            t += b
