"""Ends of what the attentions take: outputs on 16 bytes, the longest requests and one token more, hints that are too small,
more trees than are taken in the order of their length."""
import numpy as np
import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from attention_util import BF, Batch, ints, tree_masks
from gated_delta_rule_08_gb300 import binding
from layer_util import F32, HALF, f64, gen, randn, within
from oracle import attention as oracle

pytestmark = pytest.mark.gpu

LONGEST = 1 << 24


@pytest.mark.parametrize("off", [8, 16])
@pytest.mark.parametrize("d", [64, 128])
def test_outputs_on_16_bytes(off, d):
    """Walked and shared items, single tokens: rows that begin on 16 bytes but not on 32 are the same, and nothing beside them
    is written."""
    for b in (Batch([0, 90], [900, 300], H=32, Hkv=32, d=d, window=200, seed=d), Batch([3000], [100], d=d, seed=1),
              Batch([30, 7], [1, 1], d=d, seed=2)):
        want = b.run()
        room = torch.full((want.numel() + 64,), -7.0, device="cuda", dtype=BF)
        out = room[off:off + want.numel()].view_as(want)
        assert out.data_ptr() % 32 == 2 * off % 32
        b.run(out=out)
        b.check(out)
        assert torch.equal(out, want) and (room[:off] == -7).all() and (room[off + want.numel():] == -7).all()


class Long:
    """One request of `length` tokens whose table names the same few blocks again and again, as shared beginnings do."""

    def __init__(self, length, new, H=2, Hkv=1, d=64, blocks=8, seed=0):
        r = gen(seed)
        self.length, self.new, self.H, self.period = length, new, H, 256 * blocks
        self.q, (self.k, self.v) = randn(r, new, H, d, dtype=BF), (randn(r, blocks, 256, Hkv, d, dtype=BF) for _ in range(2))
        self.table = (torch.arange(-(-length // 256) + 1, device="cuda") % blocks).to(torch.int32)[None].contiguous()
        self.lengths, self.cu, self.scale = ints([length]), ints([0, new]), d ** -0.5

    def want(self, row, window, sinks):
        """(out, sum of p |v|) of a row, each key of the period with as many tokens as it stands for."""
        p = self.length - self.new + row
        times = np.zeros(self.period)
        for a, b in (((0, p + 1),) if window == 0 else ((0, min(sinks, max(0, p + 1 - window))), (max(0, p + 1 - window), p + 1))):
            times += (b - a) // self.period
            at = np.arange(a, a + (b - a) % self.period) % self.period
            np.add.at(times, at, 1)
        k, v = (f64(c).reshape(self.period, -1) for c in (self.k, self.v))
        s = self.scale * f64(self.q[row]) @ k.T
        w = np.where(times > 0, times * np.exp(s - s.max(1, keepdims=True)), 0.0)
        w /= w.sum(1, keepdims=True)
        return w @ v, w @ np.abs(v)

    def check(self, out, rows, window, sinks, inner):
        assert kda.kda_get_device_error() == 0
        for row in rows:
            want, mag = self.want(row, window, sinks)
            within(out[row], want, HALF[BF] * (np.abs(want) + inner * mag) + inner * mag, row)


@pytest.mark.parametrize("new", [1, 30, 700])
def test_a_window_at_the_end_of_the_longest_request(new):
    """Weights to bf16, and fp32 sums of some 400 products and exponentials (the bound of Batch.check)."""
    r = Long(LONGEST, new, seed=new)
    out = kda.kda_window_attention_fwd(r.q, r.k, r.v, r.table, r.lengths, r.cu, window=333, sinks=70)
    r.check(out, range(0, new, max(1, new // 40)), 333, 70, HALF[BF] + 4 * F32 * (2 * 68 * 16 + 420))
    if new == 1:
        step = kda.kda_window_attention_decode_step(r.q, r.k, r.v, r.table, r.lengths, window=333, sinks=70)
        r.check(step, [0], 333, 70, HALF[BF] + 4 * F32 * (2 * 68 * 16 + 420))


@pytest.mark.parametrize("new,H", [(1, 2), (19712, 1)])
def test_all_keys_of_the_longest_request(new, H):
    """The longest that a role of the kernels waits for another, by itself and in items of a walk.  The products' sums take 2^20
    steps, each off by at most 2^-23 of the magnitudes (it may be truncated), the weights' 2^17 of 2^-24."""
    r = Long(LONGEST, new, H=H, seed=3)
    out = kda.kda_window_attention_fwd(r.q, r.k, r.v, r.table, r.lengths, r.cu)
    r.check(out, [0] if new == 1 else [0, 100, 9999, 19711], 0, 0, HALF[BF] + 2.0 ** -3 + 2.0 ** -7)


@pytest.mark.parametrize("new", [1, 700])
def test_longer_requests_are_refused(new):
    for length in (LONGEST + 1, LONGEST + 256):
        r = Long(length, new, seed=4)
        out = torch.full_like(r.q, -7.0)
        kda.kda_window_attention_fwd(r.q, r.k, r.v, r.table, r.lengths, r.cu, out=out, window=50)
        assert kda.kda_get_device_error() == binding.DEVERR_BAD_SEQLENS and (out == -7).all()
        if new == 1:
            kda.kda_window_attention_decode_step(r.q, r.k, r.v, r.table, r.lengths, out=out, window=50)
            assert kda.kda_get_device_error() == binding.DEVERR_BAD_SEQLENS and (out == -7).all()


@pytest.mark.parametrize("hint", [1, 100, 10 ** 9])
def test_hints_cost_time_only(hint):
    for b in (Batch([3000], [100], seed=5), Batch([900, 0], [300, 700], H=32, Hkv=32, d=64, seed=6),
              Batch([5000, 40, 700], [60, 64, 3], H=32, Hkv=8, seed=7, masks=[tree_masks(n, n) for n in (60, 64, 3)]),
              Batch([4000], [12], seed=8, masks=[tree_masks(12, 1)])):
        b.check(b.run(max_length=hint))


@pytest.mark.parametrize("N", [64, 65, 90])
def test_many_trees_of_cut_requests(N):
    """Up to 64 requests are taken by falling length, more as they come; in both, long ones are cut."""
    new = [1 + (i * 5) % 40 for i in range(N)]
    before = [9000 if i % 30 == 7 else (i * 53) % 700 for i in range(N)]
    b = Batch(before, new, H=16, Hkv=2, d=64, block=64, window=0, seed=N, masks=[tree_masks(n, i) for i, n in enumerate(new)])
    b.check(b.run())
