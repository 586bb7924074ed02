"""Rotary angles of high frequencies at far positions, where a position times a frequency has many whole turns."""
import numpy as np
import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from attention_util import BF
from layer_util import F32, HALF, f64, gen, randn, within
from oracle import attention as oracle

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_high_frequencies_at_far_positions(interleaved, sign):
    """The angle is off by less than 2^-25 of a turn for frequencies up to 64, cosine, sine and sums by a few F32, then one
    rounding to bf16."""
    T, d, r = 400, 64, gen(1)
    q, k = randn(r, T, 3, d), randn(r, T, 1, d)
    freq = sign * torch.logspace(-30, 6, d // 2, base=2.0, device="cuda", dtype=torch.float64)
    pos = torch.randint(-2 ** 31, 2 ** 31, (T,), generator=r, device="cuda").to(torch.int32)
    pos[:4] = torch.tensor([0, 1, -2 ** 31, 2 ** 31 - 1], device="cuda", dtype=torch.int32)
    cache = [torch.zeros(T // 16, 16, 1, d, device="cuda", dtype=BF) for _ in range(2)]
    slot = torch.arange(T, device="cuda", dtype=torch.int32)
    out = kda.kda_rope_append(q, k, k, freq, pos, slot, *cache, interleaved=interleaved)
    assert kda.kda_get_device_error() == 0
    for got, x in ((out, q), (cache[0].view(T, 1, d), k)):
        want = oracle.rotate(f64(x), pos.cpu().numpy()[None], f64(freq), [0] * (d // 2), interleaved)
        size = np.sqrt(2) * np.abs(f64(x)).max(-1, keepdims=True)
        within(got, want, HALF[BF] * np.abs(want) + (2 * np.pi * 2.0 ** -25 + 16 * F32) * size, "rotated")
