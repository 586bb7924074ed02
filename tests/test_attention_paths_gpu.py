"""Paths of the attention kernels that depend on sizes: CTAs that walk over several items, clusters that share one,
requests cut by their own length, tiles whose halves see different keys; and waits that run out."""
import time

import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from attention_util import BF, Batch, ints, mask_words, tree_masks
from gated_delta_rule_08_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,Hkv,d,block", [(32, 32, 64, 16), (32, 32, 128, 64), (40, 8, 128, 32), (36, 12, 64, 128), (32, 16, 128, 256)])
@pytest.mark.parametrize("view", [(0, 0), (200, 6), (17, 150)])
def test_prompts_of_more_items_than_ctas(H, Hkv, d, block, view):
    """180 to 340 items on 152 SMs: barriers, stages, phases and staging go on from item to item, over requests of every
    length, some without new tokens."""
    b = Batch([0, 300, 0, 77, 5], [700, 130, 0, 900, 1], H=H, Hkv=Hkv, d=d, block=block, window=view[0], sinks=view[1], seed=H + d)
    b.check(b.run())


@pytest.mark.parametrize("n", [31, 32, 33, 65])
def test_many_short_prompts(n):
    """Requests past one look of a warp at the offsets."""
    new = [1 + (7 * i) % 90 for i in range(n)]
    b = Batch([(13 * i) % 40 for i in range(n)], new, H=16, Hkv=4, d=64, window=30, sinks=2, seed=n)
    b.check(b.run())


def test_a_long_prompt_with_a_window_and_one_without():
    for window, sinks in ((1024, 4), (0, 0)):
        b = Batch([500], [3500], H=8, Hkv=2, block=64, window=window, sinks=sinks, seed=window)
        b.check(b.run())


def test_references_move_in_every_tile_of_a_walk():
    """Scores that rise along the keys: references are passed in most tiles, and the sums rescaled while the other half
    multiplies."""
    b = Batch([0, 0], [900, 700], H=32, Hkv=32, d=64, seed=1, poison=False)
    b.q.fill_(0.25)
    for n, step in enumerate((0.02, 0.5)):
        k = torch.arange(b.new[n], device="cuda").float()[:, None, None].mul(step).expand(-1, 32, 64).to(BF)
        at = torch.arange(b.new[n], device="cuda")
        b.k[b.table[n].long()[at // 16], at % 16] = k
        b.keys[n] = k.double().cpu().numpy()
    b.check(b.run())


@pytest.mark.parametrize("G", [17, 32, 100, 128])
def test_single_tokens_of_many_heads_a_key(G):
    """More rows than a tile of 16: the kernel for many rows, with no offsets."""
    b = Batch([700, 3, 1500, 0], [1] * 4, H=16 * G, Hkv=16, d=64, seed=G)
    b.check(b.step())


@pytest.mark.parametrize("window,sinks", [(0, 0), (300, 40)])
def test_tree_batches(window, sinks):
    """Requests of different lengths, the longest cut into parts, the order by their length."""
    before = [5000, 40, 9000, 300, 1, 700, 0, 4097]
    new = [40, 64, 33, 50, 64, 7, 12, 64]
    b = Batch(before, new, H=32, Hkv=8, window=window, sinks=sinks, block=64, seed=2, masks=[tree_masks(n, i) for i, n in enumerate(new)])
    b.check(b.run())
    b.check(b.run(max_length=9100))


def test_many_trees():
    new = [1 + i % 20 for i in range(70)]
    b = Batch([(97 * i) % 600 for i in range(70)], new, H=16, Hkv=4, seed=3, masks=[tree_masks(n, i) for i, n in enumerate(new)])
    b.check(b.run())


def test_long_requests_among_short_ones():
    b = Batch([20000, 30, 500, 7000] + [64] * 30, [1] * 34, H=8, Hkv=4, seed=4, block=128)
    b.check(b.step())


def test_captured_prompts_go_by_what_lies_on_the_device():
    b = Batch([0, 60], [400, 300], H=32, Hkv=32, d=64, seed=5)
    out = torch.zeros_like(b.q)
    want = b.run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.run(out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    b.cu.copy_(ints([0, 100, 400]))  # 300 tokens fewer are new
    out.fill_(-7)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, b.run(out=torch.full_like(out, -7.0))) and not (out[:400] == -7).all(2).any()


def test_two_streams_at_once():
    a = Batch([1000], [500], H=32, Hkv=32, d=64, seed=6)
    t = Batch([3000, 40], [20, 9], seed=7, masks=[tree_masks(20, 1), tree_masks(9, 2)])
    s = Batch([900, 4000], [1, 1], seed=8)
    calls, streams = (a.run, t.run, s.step), [torch.cuda.Stream() for _ in range(3)]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    for _ in range(10):
        got = []
        for f, stream in zip(calls, streams):
            with torch.cuda.stream(stream):
                got.append(f())
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(got, want))
    assert kda.kda_get_device_error() == 0


# ------------------------------------------------------------------ waits that run out
def kinds():
    yield "few rows", lambda: Batch([700, 30], [1, 1], seed=9)
    yield "few rows, shared", lambda: Batch([6000], [1], seed=10)
    yield "shared items", lambda: Batch([3000], [100], seed=11)
    yield "items walked over", lambda: Batch([0], [2560], H=8, Hkv=2, d=64, seed=12, window=100)
    yield "trees", lambda: Batch([3000, 5], [64, 64], H=32, Hkv=8, seed=13, masks=[tree_masks(64, i) for i in range(2)])


@pytest.mark.parametrize("what,make", list(kinds()), ids=[k for k, _ in kinds()])
@pytest.mark.parametrize("mode", ["1", "stall"])
def test_waits_that_run_out_are_reported_and_the_device_stays_usable(what, make, mode, monkeypatch):
    """With "stall" the first CTA starts no copies or no MMAs and its waits run out at their limit, about a second; the
    tile that it shares is left as it was by all that share it, and the other tiles are right."""
    b = make()
    want = b.run()
    torch.cuda.synchronize()
    out = torch.full_like(want, -7.0)
    monkeypatch.setenv("KDA_TEST_WAIT_TIMEOUT", mode)
    start = time.monotonic()
    b.run(out=out)
    torch.cuda.synchronize()
    took = time.monotonic() - start
    monkeypatch.delenv("KDA_TEST_WAIT_TIMEOUT")
    assert binding.kda_get_device_error() == binding.DEVERR_WAIT_TIMEOUT
    assert took < 10, took
    if mode == "1":
        assert (out == -7).all()
    else:
        left = (out == -7).all(2)
        assert left.any() and torch.equal(out[~left], want[~left])
        # an item's tokens, and the heads of one key head (trees, at most 64 tokens: the request's)
        G = b.H // b.Hkv
        tokens = {"few rows": 1, "few rows, shared": 1, "trees": 64}.get(what, 256 // G)
        assert int(left.sum()) <= tokens * G and int(left.any(0).sum()) == G
    for _ in range(2):
        assert torch.equal(b.run(), want)
    assert binding.kda_get_device_error() == 0
