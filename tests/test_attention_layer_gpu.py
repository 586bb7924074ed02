"""The served attention layer: block tables, rotary positions, cache, attention and projections together, against the
same layer in fp64; a prompt continued in parts, token by token and by drafted tokens; a captured step."""
import numpy as np
import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from attention_util import BF, ints, mask_words, tree_masks
from gated_delta_rule_08_gb300.attention_layer import BlockPool, WindowAttentionLayer, main
from layer_util import f64, gen, randn, rel2
from oracle import attention as oracle

pytestmark = pytest.mark.gpu

H, HKV, DH, D, WINDOW, SINKS, BLOCK = 6, 2, 64, 400, 50, 3, 16


def make(seed=1):
    r = gen(seed)
    w_qkv, w_out = randn(r, (H + 2 * HKV) * DH, D) * D ** -0.5, randn(r, D, H * DH) * (H * DH) ** -0.5
    return WindowAttentionLayer(w_qkv, w_out, H, HKV, DH, WINDOW, SINKS, norm=1 + 0.2 * randn(r, D),
                                out_norm=1 + 0.2 * randn(r, H * DH))


def plain(layer, z, positions, see):
    """The layer in fp64 on the same 8-bit weights, with no rounding between the steps, for one request's rows."""
    def norm(x, w):
        return x / np.sqrt((x * x).mean(1, keepdims=True) + layer.eps) * f64(w)

    def weight(w, s):
        n, k = np.arange(w.shape[0]) // 128, np.arange(w.shape[1]) // 128
        return f64(w) * f64(s)[n][:, k]

    row = (norm(z, layer.norm) @ weight(layer.w_qkv, layer.s_qkv).T).reshape(len(z), H + 2 * HKV, DH)
    pos, freq = np.asarray(positions)[None], f64(layer.inv_freq)
    axis = [0] * len(freq)
    q, k = (oracle.rotate(x, pos, freq, axis, False) for x in (row[:, :H], row[:, H:H + HKV]))
    o, _, _ = oracle.attention(q, k, row[:, H + HKV:], see, layer.view["scale"])
    return norm(o.reshape(len(z), -1), layer.out_norm) @ weight(layer.w_out, layer.s_out).T


def prompts(layer, lengths, x, parts=1):
    """Packed prompts of these lengths through the layer, in parts of each, on a new pool."""
    N = len(lengths)
    pool = BlockPool(N, 40, 40 * N, BLOCK)
    cache, outs = pool.cache(HKV, DH), [[] for _ in lengths]
    for c in cache:
        c.fill_(float("nan"))
    begin = np.concatenate([[0], np.cumsum(lengths)])
    for part in range(parts):
        cut = [(n * part // parts, n * (part + 1) // parts) for n in lengths]
        rows = torch.cat([x[begin[i] + a:begin[i] + b] for i, (a, b) in enumerate(cut)]).contiguous()
        step = pool.step(ints([b - a for a, b in cut]), len(rows))
        y, _ = layer.prompt(rows, rows, cache, step)
        at = 0
        for i, (a, b) in enumerate(cut):
            outs[i].append(y[at:at + b - a])
            at += b - a
    return pool, cache, torch.cat([t for o in outs for t in o])


def test_prompts_and_tokens_against_fp64():
    """Activations are rounded to e4m3 twice (at most 2^-4 of a value each, at random: 2^-4 / sqrt(3) in the 2-norm)
    and to bf16 a few times; together less than 2^-4 sqrt(2)."""
    layer, lengths = make(), (130, 1, 77)
    x = randn(gen(2), sum(lengths) + 3, D, dtype=BF)
    pool, cache, y = prompts(layer, lengths, x[:208])
    step = pool.step(ints([1, 1, 1]), 3)
    last, _ = layer.token(x[208:], x[208:], cache, step)
    at = 0
    for i, n in enumerate(lengths):
        z = 2 * f64(torch.cat([x[at:at + n], x[208 + i:209 + i]]))
        want = plain(layer, z, np.arange(n + 1), oracle.visible(n + 1, n + 1, WINDOW, SINKS))
        assert rel2(torch.cat([y[at:at + n], last[i:i + 1]]), want) <= 2.0 ** -3.5
        at += n
    assert kda.kda_get_device_error() == 0


def test_a_prompt_in_parts_and_by_tokens_is_the_same_prompt():
    """Rows of 8-bit projections, and with them keys and values, do not depend on their neighbours; what differs is the
    read-out (its weights' rounding and the order of sums: three half bf16 steps), which the second e4m3 rounding may
    widen to a step of its own."""
    layer, lengths = make(3), (200, 90)
    x = randn(gen(4), 290, D, dtype=BF)
    _, whole_cache, want = prompts(layer, lengths, x)
    _, _, y = prompts(layer, lengths, x, parts=7)
    assert rel2(y, f64(want)) <= 2.0 ** -4
    pool, cache, first = prompts(layer, (180, 70), torch.cat([x[:180], x[200:270]]))
    rows = []
    for i in range(20):
        t = torch.stack([x[180 + i], x[270 + i]])
        rows.append(layer.token(t, t, cache, pool.step(ints([1, 1]), 2))[0])
    got = torch.cat([first[:180], torch.stack([r[0] for r in rows]), first[180:], torch.stack([r[1] for r in rows])])
    assert rel2(got, f64(want)) <= 2.0 ** -4
    assert kda.kda_get_device_error() == 0


def test_drafted_tokens_are_verified_and_taken_back():
    """A tree's rows are those of the paths to its tokens; what was drafted and taken back leaves no trace."""
    layer, lengths, drafted = make(5), (100, 33), (9, 4)
    x = randn(gen(6), 133 + 13, D, dtype=BF)
    masks = [tree_masks(n, i) for i, n in enumerate(drafted)]
    pool, cache, _ = prompts(layer, lengths, x[:133])
    free = pool.free_state.clone()
    depth = [len(m) - 1 for ms in masks for m in ms]
    positions = ints([lengths[0] + d for d in depth[:9]] + [lengths[1] + d for d in depth[9:]])
    step = pool.step(ints(list(drafted)), 13)
    y, _ = layer.verify(x[133:], x[133:], cache, step, mask_words([m for ms in masks for m in ms], 1).cuda(), positions)
    at, row = 0, 0
    for i, n in enumerate(lengths):
        z = 2 * f64(torch.cat([x[at:at + n], x[133 + row:133 + row + drafted[i]]]))
        for j, m in enumerate(masks[i]):
            path = list(range(n)) + [n + k for k in sorted(m)]
            want = plain(layer, z[path], np.arange(len(path)), oracle.visible(len(path), len(path), WINDOW, SINKS))[-1:]
            assert rel2(y[row + j:row + j + 1], want) <= 2.0 ** -3
        at += n
        row += drafted[i]
    pool.step(ints([-n for n in drafted]), 0)
    assert pool.lengths.tolist() == list(lengths) and pool.free_state[1] == free[1]
    t = x[133:135]
    a, _ = layer.token(t, t, cache, pool.step(ints([1, 1]), 2))
    fresh, cache2, _ = prompts(layer, lengths, x[:133])
    b, _ = layer.token(t, t, cache2, fresh.step(ints([1, 1]), 2))
    assert torch.equal(a, b) and kda.kda_get_device_error() == 0


def test_a_captured_step_serves_token_after_token():
    layer, lengths = make(7), (40, 20)
    x = randn(gen(8), 60, D, dtype=BF)
    pool, cache, _ = prompts(layer, lengths, x)
    other, other_cache, _ = prompts(layer, lengths, x)
    counts, t = ints([1, 1]), randn(gen(9), 2, D, dtype=BF)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):  # once outside the capture, and taken back
        layer.token(t, t, cache, pool.step(counts, 2))
        pool.step(-counts, 0)
    torch.cuda.current_stream().wait_stream(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = layer.token(t, t, cache, pool.step(counts, 2))
    for i in range(30):
        new = randn(gen(100 + i), 2, D, dtype=BF)
        t.copy_(new)
        graph.replay()
        want, _ = layer.token(new, new, other_cache, other.step(counts, 2))
        assert torch.equal(y, want)
    assert pool.lengths.tolist() == [70, 50] and kda.kda_get_device_error() == 0


def test_layer_refuses_weights_of_other_heads():
    with pytest.raises(ValueError):
        WindowAttentionLayer(torch.zeros(10, 16, device="cuda"), torch.zeros(16, H * DH, device="cuda"), H, HKV, DH)


def test_the_program_runs(capsys):
    main()
    assert "drafted" in capsys.readouterr().out
