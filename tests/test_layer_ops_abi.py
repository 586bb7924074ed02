"""Refusals of the operators around a recurrent layer, and their oracle's identities (no GPU)."""
import ctypes
import os

import numpy as np
import pytest

P = ctypes.c_void_p
A, B_, C, D_, E = (P(0x1000 * i) for i in range(1, 6))
OK_WS = P(0x100000)


@pytest.fixture(scope="module")
def lib():
    from gated_delta_rule_08_gb300 import binding
    if not os.path.exists(binding.LIB_PATH):
        from gated_delta_rule_08_gb300.build import build_library
        build_library()
    return binding.load_library()


INVALID, UNSUPPORTED, WORKSPACE = 1, 2, 5


def norm(lib, x=A, r=None, w=None, rout=None, y=B_, s=C, rows=4, D=256, eps=1e-6, dt=0):
    return lib.kda_rmsnorm_quant(x, r, w, rout, y, s, rows, D, eps, dt, None)


def test_rmsnorm_quant_refuses(lib):
    assert norm(lib, rows=-1) == INVALID and norm(lib, D=0) == INVALID and norm(lib, eps=-1.0) == INVALID
    assert norm(lib, eps=float("nan")) == INVALID
    assert norm(lib, D=250) == UNSUPPORTED and norm(lib, D=32784) == UNSUPPORTED and norm(lib, dt=2) == UNSUPPORTED
    assert norm(lib, x=None) == INVALID and norm(lib, y=None) == INVALID and norm(lib, s=None) == INVALID
    assert norm(lib, rout=D_) == INVALID                      # a sum's output without a residual
    assert norm(lib, y=A) == INVALID and norm(lib, r=B_) == INVALID
    assert norm(lib, x=P(0x1008)) == INVALID and norm(lib, w=P(0x5004)) == INVALID and norm(lib, s=P(0x3002)) == INVALID


def matmul(lib, a=A, sa=B_, b=C, sb=D_, out=E, M=4, N=4, K=64, dt=0):
    return lib.kda_matmul_fp8(a, sa, b, sb, out, M, N, K, dt, None)


def test_matmul_fp8_refuses(lib):
    assert matmul(lib, M=-1) == INVALID and matmul(lib, N=0) == INVALID and matmul(lib, K=0) == INVALID
    assert matmul(lib, K=40) == UNSUPPORTED and matmul(lib, dt=3) == UNSUPPORTED and matmul(lib, M=(1 << 22) + 1) == UNSUPPORTED
    for name in ("a", "sa", "b", "sb", "out"):
        assert matmul(lib, **{name: None}) == INVALID
    assert matmul(lib, out=A) == INVALID and matmul(lib, out=D_) == INVALID
    assert matmul(lib, a=P(0x1008)) == INVALID and matmul(lib, sb=P(0x4002)) == INVALID


def chunk(lib, q=A, k=B_, v=C, g=D_, h0=None, cu=None, out=E, hT=None, B=1, T=64, H=2, dk=128, dv=128, qs=256, ks=256,
          vs=256, dt=0, odt=0, ws=OK_WS, nbytes=1 << 40):
    return lib.kda_linear_chunk_fwd(q, k, v, g, 1, h0, cu, out, hT, B, T, H, dk, dv, qs, ks, vs, 1.0, dt, odt, ws, nbytes,
                                    None)


def test_linear_chunk_refuses(lib):
    assert chunk(lib, B=0) == INVALID and chunk(lib, T=-1) == INVALID and chunk(lib, H=0) == INVALID
    assert chunk(lib, dk=96) == UNSUPPORTED and chunk(lib, dv=32) == UNSUPPORTED and chunk(lib, dt=2) == UNSUPPORTED
    assert chunk(lib, odt=5) == UNSUPPORTED and chunk(lib, T=1 << 31) == UNSUPPORTED and chunk(lib, B=1 << 20, T=1 << 30) == UNSUPPORTED
    assert chunk(lib, B=16385, cu=P(0x7000)) == UNSUPPORTED and chunk(lib, cu=P(0x7002)) == INVALID
    assert chunk(lib, qs=255) == INVALID      # rows overlap
    assert chunk(lib, ks=260) == INVALID      # a row off the 16-byte boundary
    assert chunk(lib, vs=1 << 33) == INVALID
    for name in ("q", "k", "v", "g", "out"):
        assert chunk(lib, **{name: None}) == INVALID
    assert chunk(lib, out=C) == INVALID and chunk(lib, q=P(0x1008)) == INVALID and chunk(lib, hT=P(0x9004)) == INVALID
    assert chunk(lib, ws=None) == WORKSPACE and chunk(lib, nbytes=16) == WORKSPACE and chunk(lib, ws=P(0x100010)) == WORKSPACE


def step(lib, q=A, k=B_, v=C, g=D_, pool=P(0x8000), slot=P(0x9000), out=E, N=4, H=2, dk=128, dv=128, slots=8, qs=256,
         ks=256, vs=256, dt=0, odt=0):
    return lib.kda_linear_decode_step(q, k, v, g, 0, pool, slot, out, N, H, dk, dv, slots, qs, ks, vs, 1.0, dt, odt, None)


def test_linear_step_refuses(lib):
    assert step(lib, N=-1) == INVALID and step(lib, H=0) == INVALID and step(lib, slots=-1) == INVALID
    assert step(lib, dk=32) == UNSUPPORTED and step(lib, odt=2) == UNSUPPORTED and step(lib, N=1 << 30) == UNSUPPORTED
    for name in ("q", "k", "v", "g", "pool", "slot", "out"):
        assert step(lib, **{name: None}) == INVALID
    assert step(lib, qs=128) == INVALID and step(lib, vs=257) == INVALID and step(lib, pool=P(0x8008)) == INVALID


def test_linear_workspace_size(lib):
    f = lib.kda_linear_chunk_fwd_workspace_size
    assert f(1, 8192, 32, 128, 128, 0) > 0 and f(1, 0, 1, 64, 64, 1) > 0
    assert f(0, 8192, 32, 128, 128, 0) == 0 and f(1, -1, 32, 128, 128, 0) == 0 and f(1, 64, 1, 100, 128, 0) == 0
    assert f(1, 64, 1, 128, 128, 2) == 0


def test_binding_refuses_host_tensors_and_wrong_types():
    import torch
    import gated_delta_rule_08_gb300 as kda
    x = torch.zeros(2, 64)
    with pytest.raises(ValueError):
        kda.kda_rmsnorm_quant(x)
    with pytest.raises(TypeError):
        kda.kda_rmsnorm_quant(x.half())
    with pytest.raises(ValueError):
        kda.kda_matmul_fp8(x.to(torch.float8_e4m3fn), x, x.to(torch.float8_e4m3fn), x)
    q = torch.zeros(2, 2, 64)
    with pytest.raises(ValueError):
        kda.kda_linear_decode_step(q, q, q, torch.zeros(2), torch.zeros(4, 2, 64, 64), torch.zeros(2, dtype=torch.int32))


# ------------------------------------------------------------------ the oracle
def test_recurrence_is_the_masked_sum():
    """o_i = scale * sum_{j <= i} e^{g_{j+1} + .. + g_i} (q_i . k_j) v_j, and from h0 e^{g_1 + .. + g_i} h0^T q_i."""
    from oracle.layer import linear_recurrence
    r = np.random.default_rng(1)
    T, H, dk, dv = 7, 2, 3, 4
    q, k, v, g = r.normal(size=(T, H, dk)), r.normal(size=(T, H, dk)), r.normal(size=(T, H, dv)), -r.random((T, H))
    h0 = r.normal(size=(1, H, dk, dv))
    out, S, mag, M = linear_recurrence(q, k, v, g, h0=h0, scale=0.5)
    G = np.cumsum(g, 0)
    for h in range(H):
        for i in range(T):
            o = np.exp(G[i, h]) * q[i, h] @ h0[0, h]
            for j in range(i + 1):
                o = o + np.exp(G[i, h] - G[j, h]) * (q[i, h] @ k[j, h]) * v[j, h]
            np.testing.assert_allclose(out[i, h], 0.5 * o, rtol=1e-12, atol=1e-13)
    assert (mag >= np.abs(out) * (1 - 1e-12)).all() and (M >= np.abs(S) * (1 - 1e-12)).all()


def test_recurrence_resets_and_packs():
    from oracle.layer import linear_recurrence
    r = np.random.default_rng(2)
    T, H, d = 6, 1, 2
    q, k, v, g = (r.normal(size=(T, H, d)) for _ in range(4))
    g = -np.abs(g[..., 0])
    g[3] = -np.inf  # the same as a new sequence from token 3 on
    out, S, _, _ = linear_recurrence(q, k, v, g)
    out2, S2, _, _ = linear_recurrence(q, k, v, g, cu=[0, 3, 3, 6])
    np.testing.assert_array_equal(out, out2)
    np.testing.assert_array_equal(S[0], S2[2])
    assert not S2[1].any()


def test_blocks_of_the_norm_and_product():
    from oracle.layer import block_matmul, rmsnorm_blocks
    r = np.random.default_rng(3)
    x = r.normal(size=(3, 200))
    x[1] = 0
    z, ratio, scale = rmsnorm_blocks(x, None, None, 1e-6)
    assert np.allclose(np.abs(ratio[0, :128]).max(), 448) and np.allclose(np.abs(ratio[0, 128:]).max(), 448)
    assert not ratio[1].any() and (scale[1] == 1e-30 / 448).all()
    y = ratio * scale[:, np.arange(200) // 128]
    np.testing.assert_allclose((y[0] ** 2).mean(), 1, rtol=1e-5)
    out, mag = block_matmul(ratio, scale, ratio, scale[:1])
    np.testing.assert_allclose(out[:1], y[:1] @ (ratio * scale[:1, np.arange(200) // 128]).T, rtol=1e-12)
    assert (mag >= np.abs(out) * (1 - 1e-12)).all()
