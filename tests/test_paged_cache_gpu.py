"""Block tables against a list of blocks, and rotary positions with the cache's write against complex numbers."""
import numpy as np
import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from attention_util import BF, ints
from gated_delta_rule_08_gb300 import binding
from layer_util import F32, HALF, f64, gen, randn, within
from oracle import attention as oracle

pytestmark = pytest.mark.gpu


class Pool:
    """Requests on a pool of blocks, on the device and as lists."""

    def __init__(self, N, width, blocks, block, head=0, seed=0):
        r = np.random.default_rng(seed)
        self.block, self.blocks = block, blocks
        self.free = r.permutation(blocks).tolist()
        self.lengths, self.rows = [0] * N, [[-1] * width for _ in range(N)]
        ring = np.full(blocks, -1)
        ring[(head + np.arange(blocks)) % blocks] = self.free
        self.ring, self.state = ints(ring.tolist()), ints([head, blocks])
        self.table = torch.full((N, width), -1, dtype=torch.int32, device="cuda")
        self.dev_lengths = ints(self.lengths)

    def step(self, counts, room=0, in_place=True):
        T = sum(max(c, 0) for c in counts) + room
        want = oracle.block_tables(counts, self.lengths, self.rows, self.free, self.block, T, self.blocks)
        own = dict(new_lengths=self.dev_lengths, new_free_state=self.state) if in_place else {}
        slot, pos, cu, lengths, state = kda.kda_block_tables(ints(counts), self.dev_lengths, self.table, self.ring, self.state,
                                                            block_size=self.block, max_tokens=T, **own)
        assert kda.kda_get_device_error() == 0
        slots, positions, offsets, self.lengths, self.rows, self.free = want
        assert slot.tolist() == slots and pos.tolist() == positions and cu.tolist() == offsets
        assert lengths.tolist() == self.lengths and self.table.tolist() == self.rows
        head, free = state.tolist()
        ring = self.ring.tolist()
        assert free == len(self.free) and [ring[(head + i) % self.blocks] for i in range(free)] == self.free
        self.dev_lengths, self.state = lengths, state


@pytest.mark.parametrize("block", [16, 64, 256])
@pytest.mark.parametrize("in_place", [True, False])
def test_steps_of_a_pool(block, in_place):
    """Prompts, single tokens, drafted tokens taken back, ends and new beginnings, until the ring has come round."""
    r = np.random.default_rng(block)
    p = Pool(37, 9, 150, block, head=140, seed=1)
    for step in range(25):
        counts = []
        for n, a in enumerate(p.lengths):
            kind = r.integers(0, 5)
            most = 4 * block
            counts.append(int({0: 0, 1: 1, 2: min(int(r.integers(0, most)), 9 * block - a) if a < 2 * block else -int(r.integers(0, a + 1)),
                               3: -a, 4: -min(a, 5)}[int(kind)]))
            if a + counts[-1] > 9 * block:
                counts[-1] = 0
        p.step(counts, room=int(r.integers(0, 9)), in_place=in_place)


@pytest.mark.parametrize("N,count,room", [(1, 1, 0), (1, 0, 0), (1, 20000, 3), (3, 7000, 0), (1024, 1, 0), (1025, 9, 1), (8192, 1, 0)])
def test_sizes(N, count, room):
    p = Pool(N, -(-count // 16) + 1, N * (-(-count // 16) + 1), 16, head=5 % N, seed=N)
    p.step([count] * N, room)
    p.step([max(0, 3 - i % 5) for i in range(N)], room)
    p.step([-a if i % 2 else 0 for i, a in enumerate(p.lengths)], room)


def test_no_requests_and_no_tokens():
    p = Pool(0, 4, 8, 16)
    slot, pos, cu, lengths, state = kda.kda_block_tables(ints([]), ints([]), p.table, p.ring, p.state, block_size=16, max_tokens=3)
    assert slot.tolist() == [-1] * 3 and pos.tolist() == [0] * 3 and cu.tolist() == [0] and state.tolist() == [0, 8]
    p = Pool(2, 4, 8, 16)
    p.step([0, 0])


def refused(p, counts, bits, max_tokens=1000, **change):
    before = [t.clone() for t in (p.table, p.ring)]
    lengths, state = change.get("lengths", p.dev_lengths), change.get("state", p.state)
    slot, pos, cu, new, left = kda.kda_block_tables(ints(counts), lengths, p.table, p.ring, state, block_size=p.block,
                                                    max_tokens=max_tokens)
    assert kda.kda_get_device_error() == bits
    assert (slot == -1).all() and not pos.any() and not cu.any()
    assert torch.equal(new, lengths) and torch.equal(left, state)
    assert torch.equal(p.table, before[0]) and torch.equal(p.ring, before[1])


def test_steps_that_do_nothing():
    p = Pool(3, 4, 6, 16, seed=2)
    p.step([20, 16, 1])
    refused(p, [60, 0, 0], binding.DEVERR_BAD_COUNT)            # past the row
    refused(p, [0, -17, 0], binding.DEVERR_BAD_COUNT)           # below 0
    refused(p, [2 ** 31 - 1, 0, 0], binding.DEVERR_BAD_COUNT)
    refused(p, [-2 ** 31, 0, 0], binding.DEVERR_BAD_COUNT)
    refused(p, [5, 5, 5], binding.DEVERR_BAD_COUNT, max_tokens=14)
    refused(p, [12, 32, 31], binding.DEVERR_NO_BLOCKS)          # two blocks are free, three needed
    refused(p, [12, 32, 31, ][:3], binding.DEVERR_NO_BLOCKS, max_tokens=9000)
    refused(p, [1, 1, 1], binding.DEVERR_BAD_COUNT, lengths=ints([-1, 16, 1]))
    refused(p, [1, 1, 1], binding.DEVERR_BAD_COUNT, state=ints([6, 2]))
    refused(p, [1, 1, 1], binding.DEVERR_BAD_COUNT, state=ints([0, 7]))
    refused(p, [-20, 0, 0], binding.DEVERR_BAD_COUNT, state=ints([0, 5]))  # more blocks than there are
    p.step([1, 1, 1])


def test_blocks_outside_the_pool_are_reported():
    p = Pool(2, 4, 6, 16, seed=3)
    p.step([20, 3])
    p.table[1, 0] = 99
    slot, *_ = kda.kda_block_tables(ints([1, 2]), p.dev_lengths, p.table, p.ring, p.state, block_size=16, max_tokens=3)
    assert kda.kda_get_device_error() == binding.DEVERR_BAD_SLOT
    assert slot[0] >= 0 and slot[1:].tolist() == [-1, -1]


def test_a_captured_step_goes_on():
    """In place, a replayed step counts on."""
    p, q = Pool(5, 6, 30, 16, seed=4), Pool(5, 6, 30, 16, seed=4)
    counts = ints([1] * 5)
    slot = torch.empty(5, dtype=torch.int32, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kda.kda_block_tables(counts, p.dev_lengths, p.table, p.ring, p.state, block_size=16, max_tokens=5,
                             new_lengths=p.dev_lengths, new_free_state=p.state, slot_map=slot)
    for _ in range(40):
        graph.replay()
        q.step([1] * 5)
    torch.cuda.synchronize()
    assert torch.equal(p.table, q.table) and torch.equal(p.state, q.state) and p.dev_lengths.tolist() == [40] * 5


# ------------------------------------------------------------------ rotary positions
def rope_case(seed, T, H, Hkv, d, rot, axes, dtype, far, block=16, packed=False, layout="token", interleaved=False, skip=()):
    r = gen(seed)
    if packed:
        row = randn(r, T, (H + 2 * Hkv) * d + 8, dtype=dtype)[:, :(H + 2 * Hkv) * d].view(T, H + 2 * Hkv, d)
        q, k, v = row[:, :H], row[:, H:H + Hkv], row[:, H + Hkv:]
    else:
        q, k, v = (randn(r, T, n, d, dtype=dtype) for n in (H, Hkv, Hkv))
    n = rot // 2
    freq = 10000.0 ** (-torch.arange(n, device="cuda", dtype=torch.float64) / max(n, 1))
    axis = (torch.arange(n, device="cuda") % axes).to(torch.int32)
    pos = torch.randint(-far if far > 5000 else 0, far, (axes, T), generator=r, device="cuda", dtype=torch.int32)
    blocks = -(-T // block) + 2
    slot = torch.randperm(blocks * block, generator=r, device="cuda")[:T].to(torch.int32)
    for i in skip:
        slot[i] = -1
    shape = (blocks, Hkv, block, d) if layout == "head" else (blocks, block, Hkv, d)
    caches = [randn(r, *shape, dtype=BF) for _ in range(2)]
    if layout == "head":
        caches = [c.transpose(1, 2) for c in caches]
    old = [c.clone() for c in caches]
    out = torch.full((T, H, d), -7.0, device="cuda", dtype=BF)
    got = kda.kda_rope_append(q, k, v, freq, pos if axes > 1 else pos[0], slot, *caches, axis=axis if axes > 1 else None,
                              interleaved=interleaved, q_out=out)
    assert got is out and kda.kda_get_device_error() == 0
    args = (pos.cpu().numpy(), f64(freq), axis.tolist(), interleaved)
    live = (slot >= 0).cpu().numpy()

    def near(got, x):
        """The angle is off by at most 2^-24 turns or so (its rounding to fp32; the frequency's, times the position),
        cosine and sine by a few F32, the sums by two more, then one rounding to bf16."""
        want = oracle.rotate(f64(x), *args)
        size = np.sqrt(2) * np.abs(f64(x)).max(-1, keepdims=True)
        within(got, want, HALF[BF] * np.abs(want) + (2 * np.pi * 2.0 ** -24 + 16 * F32) * size, "rotated")

    near(out[slot >= 0], q[slot >= 0]) if live.all() else None
    if not live.all():
        args = (args[0][:, live], *args[1:])
        near(out[slot >= 0], q[slot >= 0])
    assert (out[slot < 0] == -7).all()
    at = slot[slot >= 0].long()
    near(caches[0][at // block, at % block], k[slot >= 0])
    assert torch.equal(caches[1][at // block, at % block], v[slot >= 0].to(BF))
    for c, o in zip(caches, old):  # nothing else has changed
        o[at // block, at % block] = c[at // block, at % block]
        assert torch.equal(c, o)


@pytest.mark.parametrize("T", [1, 2, 5, 255, 1024, 1025, 4099])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_tokens(T, dtype):
    rope_case(T, T, 8, 2, 128, 128, 1, dtype, 5000)


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 32), (64, 16), (128, 96), (128, 128), (64, 0)])
@pytest.mark.parametrize("axes", [1, 3])
def test_rope_pairs(interleaved, d, rot, axes):
    for T in (33, 1100):
        rope_case(d + rot, T, 5, 1, d, rot, axes, BF, 5000, block=64, packed=True, interleaved=interleaved, skip=(3, 32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_rope_far_positions(dtype):
    rope_case(1, 700, 3, 3, 64, 64, 4, dtype, 2 ** 31 - 1, layout="head")


def test_rope_many_heads():
    rope_case(2, 9, 128, 1, 128, 128, 2, BF, 5000, block=256)


def test_rope_bad_slots_and_axes_are_reported():
    q, k = torch.ones(3, 2, 64, device="cuda", dtype=BF), torch.ones(3, 1, 64, device="cuda", dtype=BF)
    freq = torch.ones(32, device="cuda", dtype=torch.float64)
    for slot, axis in (([5, 64, 7], 0), ([5, -2, 7], 0), ([5, 6, 7], 1), ([5, 6, 7], -1)):
        cache, out = torch.zeros(2, 4, 16, 1, 64, device="cuda", dtype=BF), torch.full_like(q, -7.0)
        kda.kda_rope_append(q, k, k, freq, ints([1, 2, 3]), ints(slot), cache[0], cache[1], axis=ints([0] * 31 + [axis]), q_out=out)
        assert kda.kda_get_device_error() == binding.DEVERR_BAD_SLOT
        if axis == 0:
            assert (out[1] == -7).all() and not (out[[0, 2]] == -7).any() and int(cache.any(4).sum()) == 4
        else:
            assert (out == -7).all() and not cache.any()
