"""Attention over a paged cache against the fp64 oracle: prompts, single tokens, trees of drafted tokens, with windows,
sinks, every head and block layout, and NaN in all that no token sees."""
import numpy as np
import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from attention_util import BF, Batch, ints, mask_words, tree_masks
from gated_delta_rule_08_gb300 import binding

pytestmark = pytest.mark.gpu

#: window, sinks
VIEWS = {"all": (0, 0), "window": (37, 0), "sinks": (37, 5), "wide": (300, 70), "one": (1, 0), "one and sinks": (1, 17)}
#: H, Hkv, d
HEADS = {"8 of 2": (8, 2, 128), "one each": (3, 3, 64), "5 to 1": (5, 1, 128), "16 to 1": (16, 1, 64), "7 of 2": (14, 2, 64),
         "40 to 1": (40, 1, 128), "128 to 1": (128, 1, 64)}


@pytest.mark.parametrize("view", VIEWS)
@pytest.mark.parametrize("block", [16, 32, 64, 128, 256])
def test_prompts(view, block):
    w, s = VIEWS[view]
    b = Batch([0, 130, 7, 0, 500], [1, 40, 129, 300, 2], block=block, window=w, sinks=s, seed=block)
    b.check(b.run(), view)


@pytest.mark.parametrize("heads", HEADS)
@pytest.mark.parametrize("view", ["all", "sinks"])
def test_prompts_of_every_head_layout(heads, view):
    H, Hkv, d = HEADS[heads]
    w, s = VIEWS[view]
    b = Batch([0, 200, 31], [70, 33, 1], H=H, Hkv=Hkv, d=d, window=w, sinks=s, seed=3, packed=True)
    b.check(b.run(), heads)


@pytest.mark.parametrize("view", VIEWS)
@pytest.mark.parametrize("block", [16, 128, 256])
def test_single_tokens(view, block):
    w, s = VIEWS[view]
    b = Batch([0, 1, 15, 16, 17, 63, 400, 1999], [1] * 8, block=block, window=w, sinks=s, seed=block)
    out = b.step()
    b.check(out, view)
    b.check(b.run(), view)


@pytest.mark.parametrize("heads", HEADS)
def test_single_tokens_of_every_head_layout(heads):
    H, Hkv, d = HEADS[heads]
    b = Batch([900, 0, 77], [1] * 3, H=H, Hkv=Hkv, d=d, seed=4, packed=True)
    b.check(b.step(), heads)


@pytest.mark.parametrize("n,length", [(1, 1), (1, 5000), (2, 3001), (5, 1200), (40, 700), (200, 90)])
def test_single_tokens_split_and_unsplit(n, length):
    """From one request over 16 CTAs to many of one CTA each."""
    b = Batch([max(0, length - 1 - 3 * i) for i in range(n)], [1] * n, seed=n)
    b.check(b.step())
    b.check(b.step(max_length=length + 7))
    b.check(b.step(max_length=1), "a hint that is too small costs time only")


@pytest.mark.parametrize("view", VIEWS)
@pytest.mark.parametrize("block", [16, 64])
def test_trees(view, block):
    w, s = VIEWS[view]
    new = [12, 1, 64, 5]
    b = Batch([100, 0, 333, 17], new, block=block, window=w, sinks=s, seed=5, masks=[tree_masks(n, i) for i, n in enumerate(new)])
    b.check(b.run(), view)


@pytest.mark.parametrize("heads", HEADS)
def test_trees_of_every_head_layout(heads):
    H, Hkv, d = HEADS[heads]
    new = [9, 30]
    b = Batch([50, 400], new, H=H, Hkv=Hkv, d=d, seed=6, packed=True, masks=[tree_masks(n, i + 7) for i, n in enumerate(new)])
    b.check(b.run(), heads)


@pytest.mark.parametrize("n", [63, 64, 65, 130, 400])
def test_trees_of_several_mask_words(n):
    b = Batch([90, 3], [n, 2], H=4, Hkv=2, d=64, seed=8, window=100, sinks=3, masks=[tree_masks(n, 1), tree_masks(2, 2)])
    b.check(b.run())


def test_trees_with_any_mask():
    """Masks that name nothing, only others, or later tokens; a request whose rows see nothing at all gives zeros."""
    masks = [[set(), {0}, {0, 2}, {1, 3}, {4, 0}], [set(), {1}, set()]]
    b = Batch([40, 0], [5, 3], masks=masks, seed=9, window=3)
    out = b.run()
    b.check(out)
    assert not out[5].any() and not out[7].any() and out[6].any()


def test_a_chain_of_drafted_tokens_is_a_prompt():
    new = [20, 3]
    chain = [[set(range(i + 1)) for i in range(n)] for n in new]
    b = Batch([70, 5], new, window=50, sinks=4, seed=10, masks=chain)
    a = b.run()
    b.check(a)
    b.masks = None
    b.check(b.run())


@pytest.mark.parametrize("layout", ["token", "head"])
@pytest.mark.parametrize("d", [64, 128])
def test_cache_layouts(layout, d):
    b = Batch([45, 200], [30, 1], d=d, layout=layout, seed=11, block=32)
    b.check(b.run())


def test_caches_that_are_parts_of_one_tensor():
    b = Batch([45, 200], [30, 1], seed=12, block=32)
    both = torch.stack([b.k, b.v], 1)  # [blocks, 2, block, Hkv, d]
    b.k, b.v = both[:, 0], both[:, 1]
    b.check(b.run())


def test_one_block_of_one_head_and_one_token():
    b = Batch([0], [1], H=1, Hkv=1, d=64, seed=13, spare=0)
    b.check(b.run())
    b.check(b.step())


@pytest.mark.parametrize("size", [1e-3, 30.0])
def test_scores_near_zero_and_far_apart(size):
    """Weights that are all alike, and weights of which one is nearly all, with references that move many times."""
    b = Batch([700, 64], [140, 1], H=4, Hkv=2, seed=14, scale=size * 128 ** -0.5)
    b.check(b.run())


def test_rising_scores():
    """Each key scores above the ones before it, so that every reference is passed: by little and by far."""
    b = Batch([0, 0], [300, 280], H=2, Hkv=1, d=64, seed=15, poison=False)
    b.q.fill_(0.25)
    for n, step in enumerate((0.01, 0.5)):
        k = torch.arange(b.new[n], device="cuda").float()[:, None, None].mul(step).expand(-1, 1, 64).to(BF)
        at = torch.arange(b.new[n], device="cuda")
        pages = b.table[n].long()[at // 16]
        b.k[pages, at % 16] = k
        b.keys[n] = k.double().cpu().numpy()
    b.check(b.run())


def test_rows_behind_the_last_are_left():
    b = Batch([5, 60], [30, 2], seed=16)
    q = torch.cat([b.q, torch.full((7, 8, 128), float("nan"), device="cuda", dtype=BF)])
    out = torch.full((39, 8, 128), -7.0, device="cuda", dtype=BF)
    b.run(q=q, out=out)
    b.check(out[:32])
    assert (out[32:] == -7).all()


def test_no_tokens():
    b = Batch([5, 60], [0, 2], seed=17)
    b.check(b.run())
    b.cu = ints([0, 0, 0])
    out = torch.full((2, 8, 128), -7.0, device="cuda", dtype=BF)
    b.run(out=out)
    assert (out == -7).all()
    empty = torch.empty(0, 8, 128, device="cuda", dtype=BF)
    assert kda.kda_window_attention_fwd(empty, b.k, b.v, b.table, b.lengths, b.cu).shape == (0, 8, 128)


def test_requests_of_length_zero():
    b = Batch([5, 60, 0], [1, 1, 1], seed=18)
    b.lengths = ints([6, 0, 1])
    out = b.step()
    assert not out[1].any()
    b.see[1][:] = False
    b.check(out)


def test_bad_requests_are_skipped_and_reported():
    b = Batch([5, 60, 20], [3, 2, 1], seed=19)
    good = b.run()
    for lengths in ([8, 1, 21], [8, -5, 21], [8, 10 ** 6, 21]):  # fewer than the new tokens, negative, past the table
        out = torch.full_like(good, -7.0)
        kda.kda_window_attention_fwd(b.q, b.k, b.v, b.table, ints(lengths), b.cu, out=out, **b.options())
        assert kda.kda_get_device_error() == binding.DEVERR_BAD_SEQLENS
        assert (out[3:5] == -7).all() and torch.equal(out[:3], good[:3]) and torch.equal(out[5:], good[5:])
    for cu in ([1, 3, 5, 6], [0, 4, 3, 6], [0, 3, 5, 7]):
        out = torch.full_like(good, -7.0)
        kda.kda_window_attention_fwd(b.q, b.k, b.v, b.table, b.lengths, ints(cu), out=out, **b.options())
        assert kda.kda_get_device_error() == binding.DEVERR_BAD_SEQLENS and (out == -7).all()
    step = Batch([5, 60], [1, 1], seed=19)
    out = torch.full_like(step.q, -7.0)
    for length in (-1, 10 ** 6):
        step.lengths[0] = length
        step.step(out=out)
        assert kda.kda_get_device_error() == binding.DEVERR_BAD_SEQLENS and (out[0] == -7).all()


def test_too_many_drafted_tokens_are_reported():
    b = Batch([30, 9], [65, 2], H=2, Hkv=2, seed=20, masks=[tree_masks(65, 1), tree_masks(2, 2)])
    out = torch.full_like(b.q, -7.0)
    mask = mask_words([{0}] * 65 + [{0}, {0, 1}], 1).cuda()
    kda.kda_tree_attention(b.q, b.k, b.v, b.table, b.lengths, b.cu, mask, out=out, **b.options())
    assert kda.kda_get_device_error() == binding.DEVERR_BAD_COUNT
    assert (out[:65] == -7).all() and not (out[65:] == -7).all(2).any()


def test_blocks_outside_the_cache_are_reported_and_not_read():
    for bad in (-1, 10 ** 6):
        b = Batch([64, 20], [1, 1], seed=21)
        want = b.step()
        b.table[0, 2] = bad
        out = b.step()
        assert kda.kda_get_device_error() == binding.DEVERR_BAD_SLOT
        assert torch.equal(out[1], want[1]) and not torch.isinf(out[0].float()).any()


def test_results_repeat():
    """No atomics in the sums: equal calls give equal bits, whatever else the device runs."""
    b = Batch([3000, 10, 600], [1, 1, 1], seed=22)
    want = b.step()
    t = Batch([3000, 10], [40, 12], seed=23, masks=[tree_masks(40, 1), tree_masks(12, 2)])
    tree = t.run()
    for _ in range(5):
        assert torch.equal(b.step(), want) and torch.equal(t.run(), tree)


def test_on_another_stream_and_captured():
    b = Batch([100, 400], [1, 1], seed=24)
    want, out = b.step(), torch.zeros_like(b.q)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b.step(out=out)
    s.synchronize()
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.step(out=out)
    out.zero_()
    b.lengths -= 1  # a replay goes by what lies on the device
    graph.replay()
    torch.cuda.synchronize()
    short = b.step()
    assert torch.equal(out, short) and not torch.equal(short, want)


def test_blocks_far_into_a_large_cache():
    """Offsets past 2^32 bytes and 2^31 elements."""
    blocks = (1 << 31) // (128 * 8 * 128) + 40
    cache = torch.empty(blocks, 128, 8, 128, device="cuda", dtype=BF)
    small = Batch([300], [3], H=8, Hkv=8, block=128, seed=25, spare=0)
    far = ints([[blocks - 1, 5, blocks - 7, 0]])
    for i in range(3):
        cache[int(far[0, i])] = small.k[int(small.table[0, i])]
    values = torch.empty_like(cache)
    for i in range(3):
        values[int(far[0, i])] = small.v[int(small.table[0, i])]
    small.k, small.v, small.table = cache, values, far
    small.check(small.run())
