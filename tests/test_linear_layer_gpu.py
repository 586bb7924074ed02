"""The served linear-attention layer: the operators together, against the same layer in fp64, and a prompt that
is continued token by token against one longer prompt."""
import numpy as np
import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from gated_delta_rule_08_gb300.linear_layer import LinearAttentionLayer, block_quantize
from layer_util import f64, gen, randn, rel2
from oracle.layer import linear_recurrence

pytestmark = pytest.mark.gpu

H, DK, DV, D = 3, 64, 128, 400


def make(seed=1):
    r = gen(seed)
    w_qkv, w_out = randn(r, H * (2 * DK + DV), D) * D ** -0.5, randn(r, D, H * DV) * (H * DV) ** -0.5
    decay = torch.tensor([-0.5, -0.05, -0.005], device="cuda")
    return LinearAttentionLayer(w_qkv, w_out, H, DK, DV, decay, norm=1 + 0.2 * randn(r, D), out_norm=1 + 0.2 * randn(r, H * DV))


def plain(layer, x, lengths, h0=None):
    """The layer in fp64 on the same 8-bit weights, with no rounding between the steps."""
    def norm(z, w):
        return z / np.sqrt((z * z).mean(1, keepdims=True) + layer.eps) * f64(w)

    def weight(w, s):
        n, k = np.arange(w.shape[0]) // 128, np.arange(w.shape[1]) // 128
        return f64(w) * f64(s)[n][:, k]

    z = 2 * f64(x)
    row = norm(z, layer.norm) @ weight(layer.w_qkv, layer.s_qkv).T
    n = len(row)
    q, k = row[:, :H * DK].reshape(n, H, DK), row[:, H * DK:2 * H * DK].reshape(n, H, DK)
    o, S, _, _ = linear_recurrence(q, k, row[:, 2 * H * DK:].reshape(n, H, DV), f64(layer.log_decay), h0=h0,
                                   cu=np.concatenate([[0], np.cumsum(lengths)]), scale=layer.scale)
    return norm(o.reshape(n, -1), layer.out_norm) @ weight(layer.w_out, layer.s_out).T, z, S


def test_block_quantize():
    w = randn(gen(4), 300, 200)
    q, s = block_quantize(w)
    assert q.shape == (300, 200) and s.shape == (3, 2)
    full = q.float() * s.repeat_interleave(128, 0)[:300].repeat_interleave(128, 1)[:, :200]
    top = w.abs().amax()
    assert ((full - w).abs() <= 2.0 ** -4 * w.abs() + 2.0 ** -10 * top / 448 + 1e-6).all()


def test_prompt_and_tokens_against_fp64():
    """Activations are rounded to e4m3 twice (at most 2^-4 of a value each, at random: 2^-4 / sqrt(3) in the 2-norm)
    and to bf16 a few times; together less than 2^-4 sqrt(2)."""
    layer, lengths = make(), (130, 1, 77)
    x = randn(gen(2), sum(lengths), D, dtype=torch.bfloat16)
    cu = torch.tensor([0, 130, 131, 208], dtype=torch.int32, device="cuda")
    y, residual, states = layer.prompt(x, x, cu_seqlens=cu)
    want, z, S = plain(layer, x, lengths)
    assert rel2(y, want) <= 2.0 ** -3.5 and rel2(states, S) <= 2.0 ** -3.5 and rel2(residual, z) <= 2.0 ** -8
    pool = randn(gen(3), 8, H, DK, DV)
    slots = torch.tensor([5, 0, 2], dtype=torch.int32, device="cuda")
    pool[slots.long()] = states
    t = randn(gen(5), 3, D, dtype=torch.bfloat16)
    y, _ = layer.token(t, t, pool, slots)
    want, _, S = plain(layer, t, (1, 1, 1), h0=f64(states))
    assert rel2(y, want) <= 2.0 ** -3.5 and rel2(pool[slots.long()], S) <= 2.0 ** -3.5
    assert kda.kda_get_device_error() == 0


def test_tokens_continue_a_prompt():
    """Forty tokens at once, and thirty followed by ten single ones, see the same rows: the 8-bit rows and the projections
    are equal (a row's norm, scales and products do not depend on its neighbours), so what differs is only the
    read-out's rounding (three of half a bf16 step), which the second e4m3 rounding may widen to a step of its own."""
    layer = make(7)
    x = randn(gen(8), 40, D, dtype=torch.bfloat16)
    want, _, end = layer.prompt(x, x)
    first, _, states = layer.prompt(x[:30].contiguous(), x[:30].contiguous())
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    rows = [layer.token(x[i:i + 1].contiguous(), x[i:i + 1].contiguous(), states, slot)[0] for i in range(30, 40)]
    assert rel2(torch.cat([first] + rows), f64(want)) <= 2.0 ** -4
    assert rel2(states, f64(end)) <= 2.0 ** -14  # keys and values equal to the bit; sums in another order


def test_layer_refuses_weights_of_other_heads():
    with pytest.raises(ValueError):
        LinearAttentionLayer(torch.zeros(10, 16, device="cuda"), torch.zeros(16, H * DV, device="cuda"), H, DK, DV,
                             torch.zeros(H, device="cuda"))
