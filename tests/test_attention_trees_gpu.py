"""Drafted tokens that no row sees, as drafts padded to a fixed shape hold them: their keys, values and blocks may be anything."""
import numpy as np
import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from attention_util import Batch, mask_words, tree_masks

pytestmark = pytest.mark.gpu


def padded(drafted, live, seed):
    """A tree of `live` tokens among `drafted`, at random places; the other tokens see nothing and are seen by nobody."""
    at = sorted(np.random.default_rng(seed).choice(drafted, live, replace=False).tolist())
    masks = [set() for _ in range(drafted)]
    for i, seen in zip(at, tree_masks(live, seed)):
        masks[i] = {at[j] for j in seen}
    return masks


def poison_unseen(b):
    """NaN in what no row of its request sees, of the drafted tokens too, and -1 in the table entries of blocks that are wholly
    so."""
    for n, see in enumerate(b.see):
        length = see.shape[1]
        seen = see.any(0)
        for i in range(-(-length // b.block)):
            part = seen[i * b.block:(i + 1) * b.block]
            page = int(b.table[n, i])
            if page < 0:
                continue
            gone = torch.from_numpy(np.flatnonzero(~part)).cuda()
            for cache in (b.k, b.v):
                cache[page, gone] = float("nan")
            if not part.any():
                b.table[n, i] = -1


#: H, Hkv, d: rows of both kernels, one to several tiles of them
HEADS = [(8, 2, 128), (3, 3, 64), (16, 1, 64), (40, 1, 128), (128, 1, 64)]


@pytest.mark.parametrize("H,Hkv,d", HEADS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (30, 0), (9, 4), (1, 60)])
@pytest.mark.parametrize("block", [16, 128])
def test_padded_drafts(H, Hkv, d, window, sinks, block):
    new, live = [40, 12, 64, 50], [7, 12, 1, 0]
    b = Batch([100, 0, 333, 17], new, H=H, Hkv=Hkv, d=d, window=window, sinks=sinks, block=block, seed=1,
              masks=[padded(n, m, i) for i, (n, m) in enumerate(zip(new, live))])
    poison_unseen(b)
    b.check(b.run())


@pytest.mark.parametrize("cached", [0, 5, 3900])
@pytest.mark.parametrize("H,Hkv", [(8, 2), (32, 8)])
def test_one_padded_draft(cached, H, Hkv):
    """One request, whose keys several CTAs share: the drafted ones lie with the last of them."""
    for drafted, live in ((12, 3), (64, 5), (300, 4)):
        b = Batch([cached], [drafted], H=H, Hkv=Hkv, block=16, seed=cached, masks=[padded(drafted, live, 3)])
        poison_unseen(b)
        b.check(b.run())


def test_drafts_of_several_words_and_tiles():
    """Drafted tokens over several tiles of keys and words of the mask, of which rows see a few, and other rows others."""
    masks = [set() for _ in range(1000)]
    for i in (0, 63, 64, 127, 128, 400, 401, 640, 999):
        masks[i] = {i, (i * 7) % 1000}
    b = Batch([130, 3], [1000, 2], H=4, Hkv=2, d=64, seed=8, window=100, sinks=3, masks=[masks, tree_masks(2, 2)])
    poison_unseen(b)
    b.check(b.run())


def test_batches_of_padded_drafts():
    before = [5000, 40, 9000, 300, 1, 700, 0, 4097]
    b = Batch(before, [64] * 8, H=32, Hkv=8, block=64, seed=2, masks=[padded(64, 3 + 5 * i, i) for i in range(8)])
    poison_unseen(b)
    b.check(b.run())


def test_bits_past_a_requests_drafted_tokens_are_ignored():
    new = [12, 30, 3]
    b = Batch([50, 400, 0], new, H=8, Hkv=2, window=45, seed=6, masks=[tree_masks(n, i) for i, n in enumerate(new)])
    want = b.run()
    b.check(want)
    words = mask_words([m for ms in b.masks for m in ms], 2).cuda()
    words[:, 1] = -1
    for n, at in zip(new, (0, 12, 42)):
        words[at:at + n, 0] |= -1 << n
    got = kda.kda_tree_attention(b.q, b.k, b.v, b.table, b.lengths, b.cu, words, **b.options())
    b.check(got)
    assert torch.equal(got, want)
