"""Refusals of the attention layer's operators, and their oracle's identities (no GPU)."""
import ctypes
import os

import numpy as np
import pytest

from oracle import attention as oracle

P = ctypes.c_void_p
INVALID, UNSUPPORTED = 1, 2
STR = (ctypes.c_int64 * 3)(16 * 2 * 128, 2 * 128, 128)


def at(i):
    return P(0x1000 * i)


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_08_gb300 import binding
    if not os.path.exists(binding.LIB_PATH):
        from gated_delta_rule_08_gb300.build import build_library
        build_library()
    return binding.load_library()


def tables(lib, counts=at(1), lengths=at(2), table=at(3), ring=at(4), state=at(5), new=at(6), left=at(7), slot=at(8), pos=at(9),
           cu=at(10), N=4, width=8, blocks=32, size=16, T=4):
    return lib.kda_block_tables(counts, lengths, table, ring, state, new, left, slot, pos, cu, N, width, blocks, size, T, None)


def test_block_tables_refuses(lib):
    assert tables(lib, N=-1) == INVALID and tables(lib, width=-1) == INVALID and tables(lib, blocks=-1) == INVALID
    assert tables(lib, T=-1) == INVALID
    for size in (0, 8, 24, 512, -16):
        assert tables(lib, size=size) == UNSUPPORTED
    assert tables(lib, N=8193) == UNSUPPORTED and tables(lib, T=(1 << 30) + 1) == UNSUPPORTED
    assert tables(lib, width=1 << 30) == UNSUPPORTED and tables(lib, blocks=1 << 28) == UNSUPPORTED
    for name in ("counts", "lengths", "table", "ring", "state", "new", "left", "slot", "pos", "cu"):
        assert tables(lib, **{name: None}) == INVALID, name
        assert tables(lib, **{name: P(0x20002)}) == INVALID, name
    assert tables(lib, slot=P(0x8004)) == INVALID and tables(lib, pos=P(0x9008)) == INVALID
    assert tables(lib, new=at(1)) == INVALID and tables(lib, counts=at(2)) == INVALID


def rope(lib, q=at(1), k=at(2), v=at(3), freq=at(4), axis=at(5), pos=at(6), slot=at(7), out=at(8), kc=at(9), vc=at(10), T=4, H=4, Hkv=2,
         d=128, rot=128, axes=3, qs=512, ks=256, vs=256, blocks=8, size=16, strides=STR, dt=0):
    return lib.kda_rope_append(q, k, v, freq, axis, pos, slot, out, kc, vc, T, H, Hkv, d, rot, axes, 0, qs, ks, vs, blocks, size, strides,
                               dt, None)


def test_rope_append_refuses(lib):
    assert rope(lib, T=-1) == INVALID and rope(lib, H=0) == INVALID and rope(lib, Hkv=0) == INVALID
    assert rope(lib, rot=-16) == INVALID and rope(lib, axes=0) == INVALID and rope(lib, blocks=-1) == INVALID
    assert rope(lib, d=96) == UNSUPPORTED and rope(lib, rot=144) == UNSUPPORTED and rope(lib, rot=40) == UNSUPPORTED
    assert rope(lib, axes=5) == UNSUPPORTED and rope(lib, dt=2) == UNSUPPORTED and rope(lib, size=48) == UNSUPPORTED
    assert rope(lib, H=3) == UNSUPPORTED and rope(lib, H=258, qs=258 * 128) == UNSUPPORTED and rope(lib, T=1 << 40) == UNSUPPORTED
    assert rope(lib, qs=504) == INVALID and rope(lib, ks=260) == INVALID and rope(lib, vs=1 << 33) == INVALID
    assert rope(lib, strides=None) == INVALID and rope(lib, strides=(ctypes.c_int64 * 3)(4096, 256, 64)) == INVALID
    assert rope(lib, strides=(ctypes.c_int64 * 3)(4096, 252, 128)) == INVALID
    for name in ("q", "k", "v", "freq", "pos", "slot", "out", "kc", "vc"):
        assert rope(lib, **{name: None}) == INVALID, name
    for name in ("q", "k", "v", "out", "kc", "vc"):
        assert rope(lib, **{name: P(0x20008)}) == INVALID, name
    assert rope(lib, freq=P(0x20004)) == INVALID and rope(lib, axis=P(0x20002)) == INVALID and rope(lib, pos=P(0x20001)) == INVALID
    assert rope(lib, out=at(1)) == INVALID and rope(lib, kc=at(10)) == INVALID and rope(lib, vc=at(3)) == INVALID


def fwd(lib, q=at(1), kc=at(2), vc=at(3), table=at(4), lengths=at(5), cu=at(6), out=at(7), N=2, T=8, H=4, Hkv=2, d=128, qs=512, blocks=8,
        size=16, width=4, strides=STR, window=0, sinks=0, most=0, scale=1.0):
    return lib.kda_window_attention_fwd(q, kc, vc, table, lengths, cu, out, N, T, H, Hkv, d, qs, blocks, size, width, strides, window, sinks,
                                        most, scale, None)


def step(lib, q=at(1), kc=at(2), vc=at(3), table=at(4), lengths=at(5), out=at(7), N=2, H=4, Hkv=2, d=128, qs=512, blocks=8, size=16,
         width=4, strides=STR, window=0, sinks=0, most=0, scale=1.0):
    return lib.kda_window_attention_decode_step(q, kc, vc, table, lengths, out, N, H, Hkv, d, qs, blocks, size, width, strides, window,
                                                sinks, most, scale, None)


def tree(lib, mask=at(8), words=1, cu=at(6), q=at(1), kc=at(2), vc=at(3), table=at(4), lengths=at(5), out=at(7), N=2, T=8, H=4, Hkv=2, d=128,
         qs=512, blocks=8, size=16, width=4, strides=STR, window=0, sinks=0, most=0, scale=1.0):
    return lib.kda_tree_attention(q, kc, vc, table, lengths, cu, mask, words, out, N, T, H, Hkv, d, qs, blocks, size, width, strides, window,
                                  sinks, most, scale, None)


@pytest.mark.parametrize("call", [fwd, step, tree], ids=["fwd", "step", "tree"])
def test_attention_refuses(lib, call):
    for name in ("N", "blocks", "width", "window", "sinks", "most"):
        assert call(lib, **{name: -1}) == INVALID, name
    assert call(lib, H=0) == INVALID and call(lib, Hkv=0) == INVALID and call(lib, blocks=0) == INVALID and call(lib, width=0) == INVALID
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(lib, scale=scale) == INVALID
    assert call(lib, d=96) == UNSUPPORTED and call(lib, size=8) == UNSUPPORTED and call(lib, size=40) == UNSUPPORTED
    assert call(lib, H=5) == UNSUPPORTED and call(lib, H=258, qs=258 * 128) == UNSUPPORTED
    assert call(lib, N=1 << 21) == UNSUPPORTED and call(lib, width=1 << 30) == UNSUPPORTED and call(lib, blocks=1 << 28) == UNSUPPORTED
    assert call(lib, qs=504) == INVALID and call(lib, qs=516) == INVALID and call(lib, qs=1 << 33) == INVALID
    assert call(lib, strides=None) == INVALID and call(lib, strides=(ctypes.c_int64 * 3)(4096, 256, 120)) == INVALID
    for name in ("q", "kc", "vc", "table", "lengths", "out"):
        assert call(lib, **{name: None}) == INVALID, name
    for name in ("q", "kc", "vc", "out"):
        assert call(lib, **{name: P(0x20008)}) == INVALID, name
    assert call(lib, out=at(1)) == INVALID and call(lib, out=at(3)) == INVALID and call(lib, lengths=P(0x20002)) == INVALID


def test_packed_attention_refuses(lib):
    for call in (fwd, tree):
        assert call(lib, T=-1) == INVALID and call(lib, T=1 << 31) == UNSUPPORTED and call(lib, cu=None) == INVALID
        assert call(lib, cu=P(0x20002)) == INVALID
    assert tree(lib, mask=None) == INVALID and tree(lib, mask=P(0x20004)) == INVALID
    assert tree(lib, words=0) == INVALID and tree(lib, words=17) == UNSUPPORTED


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch
    import gated_delta_rule_08_gb300 as kda
    i = torch.zeros(2, 3, dtype=torch.int32)
    with pytest.raises(ValueError):
        kda.kda_block_tables(i[0], i[0], i, i[0], i[0], block_size=16, max_tokens=1)
    q, cache = torch.zeros(2, 2, 64, dtype=torch.bfloat16), torch.zeros(2, 16, 2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        kda.kda_window_attention_decode_step(q, cache, cache, i, i[0])
    with pytest.raises(ValueError):
        kda.kda_tree_attention(q, cache, cache, i, i[0], i[0], i)
    with pytest.raises(ValueError):
        kda.kda_rope_append(q, q, q, torch.zeros(32), i[0], i[0], cache, cache)
    with pytest.raises(TypeError):
        kda.kda_rope_append(q.half(), q, q, torch.zeros(32), i[0], i[0], cache, cache)


# ------------------------------------------------------------------ the oracle
def test_oracle_tables():
    tables = [[7, 3, -1], [-1] * 3]
    got = oracle.block_tables([5, 2], [30, 0], tables, [9, 4, 1], 16, 8, 16)
    assert got == ([3 * 16 + 14, 3 * 16 + 15, 144, 145, 146, 64, 65, -1], [30, 31, 32, 33, 34, 0, 1, 0], [0, 5, 7], [35, 2],
                   [[7, 3, 9], [4, -1, -1]], [1])
    got = oracle.block_tables([-14, 0], [30, 0], tables, [9], 16, 0, 16)
    assert got[3] == [16, 0] and got[5] == [9, 3]
    assert oracle.block_tables([0, 40], [30, 0], tables, [9, 4], 16, 99, 16) is None  # too few blocks
    assert oracle.block_tables([-31, 0], [30, 0], tables, [9], 16, 0, 16) is None
    assert oracle.block_tables([5, 2], [30, 0], tables, [9, 4, 1], 16, 6, 16) is None


def test_oracle_rotation():
    r = np.random.default_rng(0)
    x, pos = r.normal(size=(3, 2, 8)), np.array([[0, 5, -7]])
    y = oracle.rotate(x, pos, [0.5, 0.01], [0, 0], False)
    assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 4:], x[..., 4:])
    for t in range(3):
        a = pos[0, t] * 0.5
        np.testing.assert_allclose(y[t, :, 0], x[t, :, 0] * np.cos(a) - x[t, :, 2] * np.sin(a), atol=1e-14)
        np.testing.assert_allclose(y[t, :, 2], x[t, :, 2] * np.cos(a) + x[t, :, 0] * np.sin(a), atol=1e-14)
    z = oracle.rotate(x[..., [0, 2, 1, 3, 4, 5, 6, 7]], pos, [0.5, 0.01], [0, 0], True)
    np.testing.assert_allclose(z[..., [0, 2, 1, 3]], y[..., :4], atol=1e-14)
    # q . k depends on the distance alone
    q, k = r.normal(size=(1, 1, 8)), r.normal(size=(1, 1, 8))
    dots = [(oracle.rotate(q, np.array([[p + 3]]), [0.5, 0.1, 0.02, 0.3], [0] * 4, False) *
             oracle.rotate(k, np.array([[p]]), [0.5, 0.1, 0.02, 0.3], [0] * 4, False)).sum() for p in (0, 11, 10 ** 6)]
    np.testing.assert_allclose(dots, dots[0], rtol=1e-9)


def test_oracle_views():
    assert oracle.visible(5, 3, 0, 0).astype(int).tolist() == [[1, 1, 1, 0, 0], [1, 1, 1, 1, 0], [1, 1, 1, 1, 1]]
    assert oracle.visible(6, 2, 2, 1).astype(int).tolist() == [[1, 0, 0, 1, 1, 0], [1, 0, 0, 0, 1, 1]]
    chain = [{0}, {0, 1}, {0, 1, 2}]
    for w, s in ((0, 0), (7, 0), (4, 2)):
        assert np.array_equal(oracle.visible(9, 3, w, s, chain), oracle.visible(9, 3, w, s))
    assert oracle.visible(4, 2, 1, 0, [set(), {0}]).astype(int).tolist() == [[0, 1, 0, 0], [0, 0, 1, 0]]


def test_oracle_attention():
    r = np.random.default_rng(1)
    q, k, v = r.normal(size=(2, 4, 8)), r.normal(size=(6, 2, 8)), r.normal(size=(6, 2, 8))
    see = np.array([[1, 0, 1, 0, 0, 0], [0] * 6], bool)
    out, mag, _ = oracle.attention(q, k, v, see, 0.3)
    for h in range(4):
        s = np.exp(0.3 * k[[0, 2], h // 2] @ q[0, h])
        np.testing.assert_allclose(out[0, h], (s[:, None] * v[[0, 2], h // 2]).sum(0) / s.sum(), rtol=1e-12)
    assert not out[1].any() and (mag >= np.abs(out) - 1e-12).all()
