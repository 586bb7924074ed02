"""One served attention layer over a paged cache, as models put one between recurrent layers, on the library's
operators: norm with 8-bit output, 8-bit projection of q, k and v, rotary positions with the cache's write, attention with
a sliding window and sinks (prompts, single tokens, trees of drafted tokens), norm, 8-bit output projection.

    blocks = BlockPool(requests, max_blocks, num_blocks, block_size)    # tables and free blocks, for all layers
    cache = blocks.cache(Hkv, d)                                        # keys and values of one layer
    layer = WindowAttentionLayer(w_qkv, w_out, H, Hkv, d, window, sinks)

    step = blocks.step(counts, tokens)                                  # request n gains counts[n] tokens, `tokens` in all
    y, residual = layer.prompt(x, residual, cache, step)                # ... parts of prompts
    y, residual = layer.token(x, residual, cache, step)                 # ... one token of each request, or of some
    y, residual = layer.verify(x, residual, cache, step, tree_mask, positions)   # ... trees of drafted tokens
    step = blocks.step(-rejected, 0)                                    # drafted tokens taken back, requests ended

A step packs the tokens of the requests that gain some, in order of the requests; idle requests (count 0) have no row in x.
Rows of x behind the step's last token are allowed, and their results undefined.  blocks.step() by itself is one token of
every request.  Drafted tokens are taken back from the last one on: a path that is no beginning of the drafted order is
kept by taking all back and running its tokens again.

All arithmetic of a call runs in libkda; the weights are cast to 8 bits once, when the layer is made.  A step's tensors
lie on the device and are updated in place, so that a step and its layers can be captured into a graph.

Run as a program, it serves a few prompts, some tokens and some drafted tokens with random weights and prints the times:
    python -m gated_delta_rule_08_gb300.attention_layer
"""
from __future__ import annotations

from dataclasses import dataclass
from typing import Optional

import torch

from .binding import (kda_block_tables, kda_get_device_error, kda_matmul_fp8, kda_rmsnorm_quant, kda_rope_append,
                      kda_tree_attention, kda_window_attention_decode_step, kda_window_attention_fwd)
from .linear_layer import block_quantize


@dataclass
class Step:
    """What a step's layers read: slots and positions of the new tokens, where each request's begin, the tables and the
    lengths after the step."""
    slot_map: torch.Tensor
    positions: torch.Tensor
    cu_seqlens: torch.Tensor
    block_tables: torch.Tensor
    lengths: torch.Tensor
    every: bool = False  # one token of every request: row n is request n's


class BlockPool:
    """Requests on a pool of blocks of a paged cache: tables, lengths and the ring of free blocks, on the device."""

    def __init__(self, requests: int, max_blocks: int, num_blocks: int, block_size: int, device="cuda"):
        self.num_blocks, self.block_size = num_blocks, block_size
        self.block_tables = torch.full((requests, max_blocks), -1, dtype=torch.int32, device=device)
        self.lengths = torch.zeros(requests, dtype=torch.int32, device=device)
        self.free_ring = torch.arange(num_blocks, dtype=torch.int32, device=device)
        self.free_state = torch.tensor([0, num_blocks], dtype=torch.int32, device=device)
        self._ones = torch.ones_like(self.lengths)

    def cache(self, Hkv: int, d: int):
        """Keys and values of one layer, [num_blocks, block_size, Hkv, d] bf16 each."""
        shape = (self.num_blocks, self.block_size, Hkv, d)
        return tuple(torch.empty(shape, dtype=torch.bfloat16, device=self.lengths.device) for _ in range(2))

    def step(self, counts: Optional[torch.Tensor] = None, tokens: int = 0) -> Step:
        """counts: int32 [requests], tokens gained (or given up, below 0); tokens: at most so many are gained in all.  Without
        counts every request gains a token."""
        every = counts is None
        if every:
            counts, tokens = self._ones, len(self._ones)
        slot, pos, cu, _, _ = kda_block_tables(counts, self.lengths, self.block_tables, self.free_ring, self.free_state,
                                               block_size=self.block_size, max_tokens=tokens, new_lengths=self.lengths,
                                               new_free_state=self.free_state)
        return Step(slot, pos, cu, self.block_tables, self.lengths, every)


class WindowAttentionLayer:
    """w_qkv: [(H + 2 Hkv) d, D] (rows q | k | v, head after head); w_out: [D, H d]; window: tokens a token sees (0: all);
    sinks: first tokens that stay visible; inv_freq: fp64 [rot / 2] (theta 10000 over the whole head unless given), axis:
    int32 [rot / 2], each frequency's axis, or None; norms: fp32 [D] and [H d], or None (ones)."""

    def __init__(self, w_qkv: torch.Tensor, w_out: torch.Tensor, H: int, Hkv: int, d: int, window: int = 0, sinks: int = 0,
                 inv_freq: Optional[torch.Tensor] = None, axis: Optional[torch.Tensor] = None, interleaved: bool = False,
                 norm: Optional[torch.Tensor] = None, out_norm: Optional[torch.Tensor] = None, eps: float = 1e-6):
        if w_qkv.shape[0] != (H + 2 * Hkv) * d or w_out.shape[1] != H * d:
            raise ValueError("weights do not match the heads")
        self.H, self.Hkv, self.d, self.eps = H, Hkv, d, eps
        self.w_qkv, self.s_qkv = block_quantize(w_qkv)
        self.w_out, self.s_out = block_quantize(w_out)
        if inv_freq is None:
            inv_freq = 10000.0 ** (-torch.arange(d // 2, device=w_qkv.device, dtype=torch.float64) / (d // 2))
        self.inv_freq, self.axis, self.interleaved = inv_freq, axis, interleaved
        self.norm, self.out_norm = norm, out_norm
        self.view = dict(window=window, sinks=sinks, scale=d ** -0.5)

    def _q(self, x, residual, cache, step, positions):
        """Rotated queries of the new tokens, whose keys and values go to the cache."""
        y, s, residual = kda_rmsnorm_quant(x, self.norm, residual=residual, eps=self.eps)
        row = kda_matmul_fp8(y, s, self.w_qkv, self.s_qkv).view(x.shape[0], self.H + 2 * self.Hkv, self.d)  # bf16
        q, k, v = row.split((self.H, self.Hkv, self.Hkv), 1)
        q = kda_rope_append(q, k, v, self.inv_freq, step.positions if positions is None else positions, step.slot_map, *cache,
                            axis=self.axis, interleaved=self.interleaved)
        return q, residual

    def _out(self, o):
        y, s, _ = kda_rmsnorm_quant(o.view(o.shape[0], -1), self.out_norm, eps=self.eps)
        return kda_matmul_fp8(y, s, self.w_out, self.s_out)

    def prompt(self, x, residual, cache, step, positions=None):
        """x: [T, D] bf16, the step's new tokens, packed; residual: the same or None; positions: int32 [T] or [axes, T]
        (the step's unless given).  Returns (y [T, D], x + residual or None)."""
        q, residual = self._q(x, residual, cache, step, positions)
        return self._out(kda_window_attention_fwd(q, *cache, step.block_tables, step.lengths, step.cu_seqlens, **self.view)), residual

    def token(self, x, residual, cache, step, positions=None):
        """x: [T, D], one new token of each request that gains one in the step."""
        if not step.every:  # which rows are whose is on the device (256 requests of 1000 keys: 166 us of attention against 159)
            return self.prompt(x, residual, cache, step, positions)
        q, residual = self._q(x, residual, cache, step, positions)
        return self._out(kda_window_attention_decode_step(q, *cache, step.block_tables, step.lengths, **self.view)), residual

    def verify(self, x, residual, cache, step, tree_mask, positions):
        """x: [T, D], the step's new tokens, drafted as trees; tree_mask: int64 [T, words] as in kda_tree_attention;
        positions: int32 [T], each token's depth in its tree behind the request's tokens."""
        q, residual = self._q(x, residual, cache, step, positions)
        o = kda_tree_attention(q, *cache, step.block_tables, step.lengths, step.cu_seqlens, tree_mask, **self.view)
        return self._out(o), residual


def main() -> None:
    H, Hkv, d, D = 32, 8, 128, 4096
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    layer = WindowAttentionLayer(randn((H + 2 * Hkv) * d, D) * D ** -0.5, randn(D, H * d) * (H * d) ** -0.5, H, Hkv, d, window=1024,
                                 sinks=4)
    lengths = [700, 1500, 64, 3000]
    N = len(lengths)
    pool = BlockPool(N, 64, 256, 64)
    cache = pool.cache(Hkv, d)
    x = randn(sum(lengths), D).to(torch.bfloat16)

    def timed(f, n=20):
        f()
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(n):
            r = f()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / n, r

    def counts(values):
        return torch.tensor(values, dtype=torch.int32, device="cuda")

    step = pool.step(counts(lengths), sum(lengths))
    ms, (y, _) = timed(lambda: layer.prompt(x, x, cache, step))
    print(f"{N} prompts, {sum(lengths)} tokens: {ms:.3f} ms, output rms {y.float().square().mean().sqrt():.4f}")
    step = pool.step()
    t = randn(N, D).to(torch.bfloat16)
    ms, (y, _) = timed(lambda: layer.token(t, t, cache, step))
    print(f"one token of each: {ms * 1e3:.1f} us, output rms {y.float().square().mean().sqrt():.4f}")
    # seven drafted tokens of each: a root, its three children, and a child of each of them
    parents = [-1, 0, 0, 0, 1, 2, 3]
    masks, depth = [], []
    for j, parent in enumerate(parents):
        masks.append((masks[parent] if parent >= 0 else 0) | 1 << j)
        depth.append(depth[parent] + 1 if parent >= 0 else 0)
    before = pool.lengths.clone()
    step = pool.step(counts([7] * N), 7 * N)
    positions = (before[:, None] + counts(depth)).flatten()
    mask = torch.tensor(masks * N, dtype=torch.int64, device="cuda")[:, None].contiguous()
    t = randn(7 * N, D).to(torch.bfloat16)
    ms, (y, _) = timed(lambda: layer.verify(t, t, cache, step, mask, positions))
    print(f"seven drafted tokens of each: {ms * 1e3:.1f} us, output rms {y.float().square().mean().sqrt():.4f}")
    pool.step(counts([-7] * N), 0)  # none is kept
    assert torch.equal(pool.lengths, before)
    assert kda_get_device_error() == 0


if __name__ == "__main__":
    main()
