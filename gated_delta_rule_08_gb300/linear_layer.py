"""One served linear-attention layer, from the residual stream to its output projection, on the library's
operators: norm with 8-bit output, 8-bit projection of q, k and v, linear attention with one decay per head
(a prompt, or one token of each request on a pool of states), norm, 8-bit output projection.

    layer = LinearAttentionLayer(w_qkv, w_out, H, dk, dv, log_decay)
    y, residual, states = layer.prompt(x, residual, cu_seqlens=cu)      # states: [B, H, dk, dv]
    y, residual = layer.token(x, residual, state_pool, slot_idx)        # the pool's states move on by a token

All arithmetic of a call runs in libkda; the weights are cast to 8 bits once, when the layer is made.

Run as a program, it serves a few prompts and then some tokens with random weights and prints the times:
    python -m gated_delta_rule_08_gb300.linear_layer
"""
from __future__ import annotations

from typing import Optional

import torch

from .binding import (kda_get_device_error, kda_linear_chunk_fwd, kda_linear_decode_step, kda_matmul_fp8,
                      kda_rmsnorm_quant)

BLOCK = 128
FP8_MAX = 448.0


def block_quantize(w: torch.Tensor):
    """A weight [N, K] as e4m3 with one scale per 128 x 128 block, as kda_matmul_fp8 takes it."""
    N, K = w.shape
    nb, kb = -(-N // BLOCK), -(-K // BLOCK)
    wide = torch.nn.functional.pad(w.float(), (0, kb * BLOCK - K, 0, nb * BLOCK - N)).view(nb, BLOCK, kb, BLOCK)
    scale = wide.abs().amax((1, 3)).clamp_min(1e-30) / FP8_MAX
    q = (wide / scale[:, None, :, None]).clamp(-FP8_MAX, FP8_MAX).view(nb * BLOCK, kb * BLOCK)[:N, :K]
    return q.to(torch.float8_e4m3fn).contiguous(), scale.contiguous()


class LinearAttentionLayer:
    """w_qkv: [H (2 dk + dv), D] (rows q | k | v, head after head); w_out: [D, H dv]; log_decay: fp32 [H], one
    constant per head (a call may give one per token instead); norms: fp32 [D] and [H dv], or None (ones)."""

    def __init__(self, w_qkv: torch.Tensor, w_out: torch.Tensor, H: int, dk: int, dv: int, log_decay: torch.Tensor,
                 norm: Optional[torch.Tensor] = None, out_norm: Optional[torch.Tensor] = None, eps: float = 1e-6):
        self.H, self.dk, self.dv, self.eps = H, dk, dv, eps
        if w_qkv.shape[0] != H * (2 * dk + dv) or w_out.shape[1] != H * dv:
            raise ValueError("weights do not match the heads")
        self.w_qkv, self.s_qkv = block_quantize(w_qkv)
        self.w_out, self.s_out = block_quantize(w_out)
        self.log_decay, self.norm, self.out_norm = log_decay, norm, out_norm
        self.scale = dk ** -0.5

    def _qkv(self, x, residual):
        y, s, residual = kda_rmsnorm_quant(x, self.norm, residual=residual, eps=self.eps)
        row = kda_matmul_fp8(y, s, self.w_qkv, self.s_qkv)  # bf16
        n, H, dk = x.shape[0], self.H, self.dk
        q, k = (row[:, i * H * dk:(i + 1) * H * dk].view(n, H, dk) for i in (0, 1))
        return q, k, row[:, 2 * H * dk:].view(n, H, self.dv), residual

    def _out(self, o):
        y, s, _ = kda_rmsnorm_quant(o.view(o.shape[0], -1), self.out_norm, eps=self.eps)
        return kda_matmul_fp8(y, s, self.w_out, self.s_out)

    def prompt(self, x, residual=None, h0=None, cu_seqlens=None, log_decay=None):
        """x: [T_tot, D] bf16; residual: the same or None.  Returns (y [T_tot, D], x + residual or None, states after
        each sequence [B, H, dk, dv])."""
        q, k, v, residual = self._qkv(x, residual)
        g = self.log_decay if log_decay is None else log_decay
        o, states = kda_linear_chunk_fwd(q, k, v, g, h0=h0, cu_seqlens=cu_seqlens, scale=self.scale)
        return self._out(o), residual, states

    def token(self, x, residual, state_pool, slot_idx, log_decay=None):
        """x: [N, D], one token of each request; its state is state_pool[slot_idx[n]], updated in place.
        Returns (y [N, D], x + residual or None)."""
        q, k, v, residual = self._qkv(x, residual)
        g = self.log_decay if log_decay is None else log_decay
        return self._out(kda_linear_decode_step(q, k, v, g, state_pool, slot_idx, scale=self.scale)), residual


def main() -> None:
    H, dk, dv, D = 32, 128, 128, 4096
    gen = torch.Generator(device="cuda").manual_seed(0)

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    decay = -torch.pow(2.0, -8.0 * torch.arange(1, H + 1, device="cuda") / H)
    layer = LinearAttentionLayer(randn(H * (2 * dk + dv), D) * D ** -0.5, randn(D, H * dv) * (H * dv) ** -0.5, H, dk, dv, decay)
    lengths = [700, 1500, 64, 3000]
    cu = torch.tensor([sum(lengths[:i]) for i in range(len(lengths) + 1)], dtype=torch.int32, device="cuda")
    x = randn(sum(lengths), D).to(torch.bfloat16)
    pool = torch.zeros(16, H, dk, dv, device="cuda")
    slots = torch.tensor([3, 9, 0, 12], dtype=torch.int32, device="cuda")

    def timed(f, n=20):
        f()
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        for _ in range(n):
            r = f()
        b.record()
        torch.cuda.synchronize()
        return a.elapsed_time(b) / n, r

    ms, (y, residual, states) = timed(lambda: layer.prompt(x, x, cu_seqlens=cu))
    print(f"{len(lengths)} prompts, {sum(lengths)} tokens: {ms:.3f} ms, output rms {y.float().square().mean().sqrt():.4f}")
    pool[slots.long()] = states
    t = randn(len(lengths), D).to(torch.bfloat16)
    ms, (y, _) = timed(lambda: layer.token(t, t, pool, slots))
    print(f"one token of each: {ms * 1e3:.1f} us, output rms {y.float().square().mean().sqrt():.4f}")
    assert kda_get_device_error() == 0


if __name__ == "__main__":
    main()
