"""Accuracy of the states under constant decays, where every token (or chunk) is decayed by one and the same
rounded factor: its rounding must not add up over the decay's window, and the operators' states have to stay as
accurate as their sums in fp32 are."""
import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from layer_util import F32, gen, randn

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32

RATES = [-2.0 ** -8, -1.1 * 2.0 ** -8, -1e-3, -1e-4, -1e-5, -0.03, -0.3, -3.0]


def closed_form(k, v, g, h0):
    """e^{T g} h0 + sum_t e^{(T - 1 - t) g} k_t v_t^T in fp64."""
    T = k.shape[0]
    w = torch.exp(g.double()[None] * torch.arange(T - 1, -1, -1, device="cuda", dtype=torch.float64)[:, None])
    return torch.einsum("thk,thv->hkv", k.double() * w[..., None], v.double()) + torch.exp(T * g.double())[:, None, None] * h0.double()


def check(got, want, T, tokens_a_step, base):
    """The state is rounded twice at most for every token or chunk of the decay's window, half a step (F32) of its
    value each, at random: 1.5 F32 sqrt(n) in the 2-norm covers that.  `base` F32 cover what does not add up."""
    for i, rate in enumerate(RATES):
        n = min(T, -1 / rate) / tokens_a_step
        off = float((got[i].double() - want[i]).norm() / want[i].norm())
        assert off <= F32 * (base + 1.5 * n ** 0.5), (rate, off / F32, n)


@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
@pytest.mark.parametrize("T", [1024, 8192])
def test_fp32_sequences(T, dk, dv):
    """base: the decay's error over its window (a step of e^g - 1 and one of the sum) and the last token's."""
    r, H = gen(T + dk), len(RATES)
    g = torch.tensor(RATES, device="cuda")
    q, k, v, h0 = randn(r, T, H, dk), randn(r, T, H, dk), randn(r, T, H, dv), randn(r, 1, H, dk, dv)
    _, hT = kda.kda_linear_chunk_fwd(q, k, v, g, h0=h0)
    check(hT[0], closed_form(k, v, g, h0[0]), T, 1, 4)
    _, hT = kda.kda_linear_chunk_fwd(q, k, v, g.expand(T, H).contiguous(), h0=h0)
    check(hT[0], closed_form(k, v, g, h0[0]), T, 1, 4)


@pytest.mark.parametrize("copies", [1, 20], ids=["cut", "uncut"])
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 128)])
def test_bf16_sequences(dk, dv, copies):
    """base: the weights of a chunk's tokens (two steps of the exponential, half a one of the product: 5 F32) and
    the twelve accumulations of its product in the tensor core (a step each, at random: 2 sqrt(12) F32)."""
    T, H = 8192, copies * len(RATES)
    r = gen(T + dk + copies)
    g = torch.tensor(copies * RATES, device="cuda")
    q, k, v = randn(r, T, H, dk, dtype=BF), randn(r, T, H, dk, dtype=BF), randn(r, T, H, dv, dtype=BF)
    h0 = randn(r, 1, H, dk, dv)
    _, hT = kda.kda_linear_chunk_fwd(q, k, v, g, h0=h0)
    n = len(RATES)
    check(hT[0, :n], closed_form(k[:, :n], v[:, :n], g[:n], h0[0, :n]), T, 64, 12)


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_tokens_one_by_one(dtype):
    T, H, dk, dv = 2048, len(RATES), 128, 64
    r = gen(7)
    g = torch.tensor(RATES, device="cuda")
    q, k, v = randn(r, T, H, dk, dtype=dtype), randn(r, T, H, dk, dtype=dtype), randn(r, T, H, dv, dtype=dtype)
    pool = randn(r, 2, H, dk, dv)
    h0, slot = pool[1].clone(), torch.ones(1, dtype=torch.int32, device="cuda")
    for t in range(T):
        kda.kda_linear_decode_step(q[t:t + 1], k[t:t + 1], v[t:t + 1], g, pool, slot)
    check(pool[1], closed_form(k, v, g, h0), T, 1, 4)
