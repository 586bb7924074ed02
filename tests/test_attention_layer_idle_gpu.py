"""The served attention layer on a pool some of whose requests are idle: a step packs the tokens of the others."""
import numpy as np
import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from attention_util import BF, ints
from layer_util import f64, gen, randn, rel2
from oracle import attention as oracle
from test_attention_layer_gpu import D, SINKS, WINDOW, make, plain, prompts

pytestmark = pytest.mark.gpu

LENGTHS = (130, 1, 77, 33)


def check_rows(layer, x, y, lengths, tokens):
    """Row i of y is that of the token tokens[i] of request i, the last of its request; the bound is that of the test of
    prompts and tokens (two roundings to e4m3, a few to bf16)."""
    begin = np.concatenate([[0], np.cumsum(lengths)])
    for row, (n, t) in enumerate(tokens):
        z = 2 * f64(torch.cat([x[begin[n]:begin[n + 1]], t[None]]))
        want = plain(layer, z, np.arange(len(z)), oracle.visible(len(z), len(z), WINDOW, SINKS))[-1:]
        assert rel2(y[row:row + 1], want) <= 2.0 ** -3, (row, n)


@pytest.mark.parametrize("counts", [[1, 1, 0, 1], [0, 1, 1, 1], [0, 0, 0, 1], [1, 1, 1, 1]])
@pytest.mark.parametrize("room", [0, 1, 3])
def test_tokens_beside_idle_requests(counts, room):
    layer = make(11)
    x = randn(gen(12), sum(LENGTHS) + 8, D, dtype=BF)
    pool, cache, _ = prompts(layer, LENGTHS, x[:sum(LENGTHS)])
    live = [n for n, c in enumerate(counts) if c]
    t = x[sum(LENGTHS):sum(LENGTHS) + len(live) + room]
    y, residual = layer.token(t, t, cache, pool.step(ints(counts), len(t)))
    check_rows(layer, x, y, LENGTHS, [(n, t[i]) for i, n in enumerate(live)])
    assert torch.equal(residual, t + t) and kda.kda_get_device_error() == 0
    assert pool.lengths.tolist() == [a + c for a, c in zip(LENGTHS, counts)]


def test_a_request_that_has_ended_and_a_new_one():
    layer = make(13)
    x = randn(gen(14), sum(LENGTHS) + 40, D, dtype=BF)
    pool, cache, _ = prompts(layer, LENGTHS, x[:sum(LENGTHS)])
    pool.step(ints([0, 0, -77, 0]), 0)
    t = x[-3:]
    y, _ = layer.token(t, t, cache, pool.step(ints([1, 1, 0, 1]), 3))
    check_rows(layer, x, y, LENGTHS, [(0, t[0]), (1, t[1]), (3, t[2])])
    new = x[sum(LENGTHS):sum(LENGTHS) + 30]
    y, _ = layer.prompt(new, new, cache, pool.step(ints([0, 0, 30, 0]), 30))
    want = plain(layer, 2 * f64(new), np.arange(30), oracle.visible(30, 30, WINDOW, SINKS))
    assert rel2(y, want) <= 2.0 ** -3.5 and kda.kda_get_device_error() == 0


def test_a_token_of_every_request():
    """A step without counts is that of ones, in a replayed graph too."""
    layer = make(15)
    x = randn(gen(16), sum(LENGTHS) + 4, D, dtype=BF)
    pool, cache, _ = prompts(layer, LENGTHS, x[:sum(LENGTHS)])
    other, other_cache, _ = prompts(layer, LENGTHS, x[:sum(LENGTHS)])
    t = x[-4:].clone()
    y, _ = layer.token(t, t, cache, pool.step())
    check_rows(layer, x, y, LENGTHS, list(enumerate(t)))
    layer.token(t, t, other_cache, other.step(ints([1] * 4), 4))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = layer.token(t, t, cache, pool.step())
    for i in range(20):
        new = randn(gen(200 + i), 4, D, dtype=BF)
        t.copy_(new)
        graph.replay()
        want, _ = layer.token(new, new, other_cache, other.step(ints([1] * 4), 4))
        assert rel2(y, f64(want)) <= 2.0 ** -4  # (the bound between two ways to the same token)
    assert torch.equal(pool.lengths, other.lengths) and torch.equal(pool.block_tables, other.block_tables)
    assert kda.kda_get_device_error() == 0
