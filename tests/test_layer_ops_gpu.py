"""The operators around a recurrent layer against their fp64 forms, at the sizes and values where they can go wrong."""
import numpy as np
import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from gated_delta_rule_08_gb300 import binding
from layer_util import (E4M3_HALF, E4M3_TINY, F32, HALF, f64, gen, linear_bounds, linear_inputs, randn, rel2, within)
from oracle.layer import block_matmul, linear_recurrence, rmsnorm_blocks

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32
FP8 = torch.float8_e4m3fn


def no_device_error():
    assert binding.kda_get_device_error() == 0


# ------------------------------------------------------------------ norm
def check_norm(x, residual, weight, eps, got):
    y, s, z = got
    wz, ratio, scale = rmsnorm_blocks(f64(x), None if residual is None else f64(residual),
                                      None if weight is None else f64(weight), eps)
    if residual is None:
        assert z is None
    else:
        within(z, wz, (HALF[x.dtype] + 2 * F32) * np.abs(wz), "sum")
    # a thread adds up to 32 squares, then a tree of at most 10 + 32 sums; half of that relative error reaches the
    # root, whose own error, two products, the quotients and the sum z add at most 16 steps
    steps = (32 + 42) / 2 + 16
    within(s, scale, 2 * steps * F32 * scale, "scale")
    v = np.abs(ratio)
    within(y, ratio, E4M3_HALF * v * (1 + 4 * steps * F32) + E4M3_TINY + 4 * steps * F32 * v, "values")


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("rows,D", [(1, 16), (1, 4096), (5, 128), (3, 144), (130, 64), (37, 256), (33, 496), (9, 1008), (7, 2000),
                                    (4, 4112), (3, 8192), (2, 16384), (2, 16400), (1, 32768), (2050, 2080), (2100, 6000),
                                    (2048, 9008)])
@pytest.mark.parametrize("residual", [False, True], ids=["plain", "residual"])
def test_norm(rows, D, residual, dtype):
    r = gen(rows * 40000 + D)
    x = randn(r, rows, D, dtype=dtype)
    res = 3 * randn(r, rows, D, dtype=dtype) if residual else None
    w = 1 + 0.5 * randn(r, D)
    check_norm(x, res, w, 1e-6, kda.kda_rmsnorm_quant(x, w, residual=res, eps=1e-6))
    check_norm(x, res, None, 0.5, kda.kda_rmsnorm_quant(x, None, residual=res, eps=0.5))


def test_norm_in_place_and_empty():
    r = gen(7)
    x, res = randn(r, 6, 512, dtype=BF), randn(r, 6, 512, dtype=BF)
    want = kda.kda_rmsnorm_quant(x, residual=res)
    keep = res.clone()
    got = kda.kda_rmsnorm_quant(x, residual=keep, residual_out=keep)
    assert got[2] is keep
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    y, s, z = kda.kda_rmsnorm_quant(x[:0], residual=res[:0])
    assert y.shape == (0, 512) and s.shape == (0, 4) and z.shape == (0, 512)


def test_norm_of_zeros_tiny_and_huge_rows():
    x = torch.zeros(4, 256, device="cuda")
    x[1] = 1e-25
    x[2, 128:] = 3e4      # a zero block beside a large one
    x[3] = torch.linspace(-1e18, 1e18, 256)
    got = kda.kda_rmsnorm_quant(x, eps=1e-6)
    check_norm(x, None, None, 1e-6, got)
    assert not got[0][0].float().any() and not got[0][2, :128].float().any()


def test_norm_of_non_finite_rows_stays_in_the_row():
    x = torch.ones(5, 512, device="cuda", dtype=BF)
    x[1, 3] = float("nan")
    x[3, 400] = float("inf")
    y, s, _ = kda.kda_rmsnorm_quant(x)
    clean = kda.kda_rmsnorm_quant(torch.ones_like(x))
    for i in (0, 2, 4):
        assert torch.equal(y[i].view(torch.uint8), clean[0][i].view(torch.uint8)) and torch.equal(s[i], clean[1][i])
    assert torch.isnan(s[1]).any() and torch.isnan(s[3]).any()


# ------------------------------------------------------------------ product
def matmul_inputs(seed, M, N, K):
    r = gen(seed)
    kb, nb = -(-K // 128), -(-N // 128)
    a = (80 * randn(r, M, K)).clamp(-448, 448).to(FP8)
    b = (80 * randn(r, N, K)).clamp(-448, 448).to(FP8)
    return a, torch.exp(2 * randn(r, M, kb)) / 80, b, torch.exp(2 * randn(r, nb, kb)) / 80


def check_matmul(ins, out):
    want, mag = block_matmul(*(f64(t) for t in ins))
    K = ins[0].shape[1]
    # any order of K products and the blocks' scaled sums in fp32, then the output's rounding
    steps = (K + 3 * -(-K // 128) + 3) * F32
    within(out, want, HALF[out.dtype] * (np.abs(want) + steps * mag) + steps * mag, "product")
    assert rel2(out, want) <= HALF[out.dtype] + 2.0 ** -12


@pytest.mark.parametrize("M,N,K", [(1, 1, 16), (1, 128, 128), (1, 4096, 4096), (2, 130, 272), (3, 257, 2000), (8, 96, 4096),
                                   (15, 1000, 128), (16, 384, 640), (17, 333, 144), (33, 2000, 1024), (64, 640, 2048),
                                   (65, 264, 400), (100, 128, 8192), (127, 255, 1040), (128, 256, 256), (129, 129, 384),
                                   (200, 512, 96), (256, 520, 1536), (300, 1032, 2064), (513, 257, 512), (1000, 2056, 400),
                                   (1280, 2304, 256)])
@pytest.mark.parametrize("out_dtype", [BF, FP], ids=["bf16", "fp32"])
def test_matmul(M, N, K, out_dtype):
    ins = matmul_inputs(M + 7 * N + 13 * K, M, N, K)
    check_matmul(ins, kda.kda_matmul_fp8(*ins, out_dtype=out_dtype))
    no_device_error()


@pytest.mark.parametrize("M,N,K", [(129, 5001, 1040), (200, 4880, 2000), (300, 4208, 4096), (65, 12288, 2176), (1025, 1300, 2064)])
@pytest.mark.parametrize("out_dtype", [BF, FP], ids=["bf16", "fp32"])
def test_matmul_of_a_few_wide_tiles(M, N, K, out_dtype):
    """Between a quarter and half as many tiles of 128 x 256 as the device has SMs: two CTAs to a tile."""
    ins = matmul_inputs(M + N + K, M, N, K)
    check_matmul(ins, kda.kda_matmul_fp8(*ins, out_dtype=out_dtype))
    no_device_error()


def test_matmul_extreme_values_and_scales():
    """e4m3's largest and smallest numbers, scales 40 powers of two apart, zero rows, and a NaN row that
    reaches its own row of the output only."""
    M, N, K = 140, 300, 400
    a, sa, b, sb = matmul_inputs(5, M, N, K)
    a[0] = 448.0
    a[1] = 2.0 ** -9
    a[2] = 0.0
    sa[3] = 2.0 ** -40
    sa[4, 1] = 2.0 ** 40
    out = kda.kda_matmul_fp8(a, sa, b, sb, out_dtype=FP)
    check_matmul((a, sa, b, sb), out)
    assert not out[2].any()
    bad = a.clone()
    bad.view(torch.uint8)[7, 399] = 0x7F  # NaN
    got = kda.kda_matmul_fp8(bad, sa, b, sb, out_dtype=FP)
    assert torch.isnan(got[7]).all()
    rows = [i for i in range(M) if i != 7]
    assert torch.equal(got[rows], out[rows])
    few = kda.kda_matmul_fp8(bad[:9].contiguous(), sa[:9].contiguous(), b, sb, out_dtype=FP)
    assert torch.isnan(few[7]).all() and torch.isfinite(few[:7]).all() and torch.isfinite(few[8]).all()
    no_device_error()


def test_matmul_writes_nothing_outside_its_rows():
    for M, N, K in ((5, 131, 256), (150, 259, 384)):
        ins = matmul_inputs(11, M, N, K)
        buf = torch.full((M * N + 64,), -7.0, device="cuda", dtype=BF)
        out = buf[32:32 + M * N].view(M, N)
        kda.kda_matmul_fp8(*ins, out=out)
        check_matmul(ins, out)
        assert (buf[:32] == -7).all() and (buf[32 + M * N:] == -7).all()


def test_matmul_no_rows():
    a, sa, b, sb = matmul_inputs(3, 4, 64, 128)
    assert kda.kda_matmul_fp8(a[:0], sa[:0], b, sb).shape == (0, 64)


# ------------------------------------------------------------------ linear attention, sequences
def check_linear(ins, lengths, out, hT, scale):
    H, dk = ins["q"].shape[1:]
    want, S, mag, M = linear_recurrence(f64(ins["q"]), f64(ins["k"]), f64(ins["v"]), f64(ins["g"]),
                                        h0=None if ins["h0"] is None else f64(ins["h0"]),
                                        cu=np.concatenate([[0], np.cumsum(lengths)]), scale=scale)
    bo, bs = linear_bounds(max(lengths), dk, ins["q"].dtype, out.dtype, want, mag, M)
    within(out, want, bo, "out")
    if hT is not None:
        within(hT, S, bs, "state")
    if want.size > 4096:  # roundings at random: three of them for bf16 inputs, in the 2-norm
        assert rel2(out, want) <= (2.0 ** -7 if ins["q"].dtype == BF or out.dtype == BF else 1e-5)


LENGTHS = [(1,), (2,), (17,), (63,), (64,), (65,), (128,), (130,), (300,), (5, 0, 64, 1, 129), (0, 77)]


@pytest.mark.parametrize("lengths", LENGTHS, ids=[",".join(map(str, n)) for n in LENGTHS])
@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("decay,h0,packed", [("token", True, True), ("head", False, False)])
def test_linear_chunk(lengths, dtype, decay, h0, packed):
    ins = linear_inputs(sum(lengths), lengths, 3, 128, 128, dtype, decay, h0, packed)
    out, hT = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], cu_seqlens=ins["cu"], scale=0.3)
    check_linear(ins, lengths, out, hT, 0.3)
    no_device_error()


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, FP), (FP, FP), (FP, BF)])
def test_linear_chunk_dims_and_types(dk, dv, dtype, out_dtype):
    lengths = (150, 70)
    for packed in (False, True):
        ins = linear_inputs(dk + dv, lengths, 2, dk, dv, dtype, "token", True, packed)
        out, hT = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], cu_seqlens=ins["cu"],
                                           scale=dk ** -0.5, out_dtype=out_dtype)
        assert out.dtype == out_dtype
        check_linear(ins, lengths, out, hT, dk ** -0.5)


@pytest.mark.parametrize("H,T", [(1, 3000), (2, 2500), (40, 700)])
def test_linear_chunk_long(H, T):
    """Few long sequences, which are split over the device, and many heads, which are not."""
    for decay in ("token", "head"):
        ins = linear_inputs(T, (T,), H, 128, 128, BF, decay, True, True)
        out, hT = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], scale=0.1)
        check_linear(ins, (T,), out, hT, 0.1)
    no_device_error()


@pytest.mark.parametrize("lengths", [(832,), (833,), (1000,), (1025,), (2000, 300, 0, 65), (64, 1500, 900)],
                         ids=lambda n: ",".join(map(str, n)))
@pytest.mark.parametrize("H", [2, 32])
def test_linear_chunk_short_segments(lengths, H):
    """Lengths around the shortest ones that are cut, and cut ones beside others that end in their first segment."""
    ins = linear_inputs(H + sum(lengths), lengths, H, 128, 128, BF, "token", True, True)
    out, hT = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], cu_seqlens=ins["cu"], scale=0.1)
    check_linear(ins, lengths, out, hT, 0.1)
    no_device_error()


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_linear_chunk_decay_extremes(dtype):
    """No decay at all, decays that empty the state in a token (-inf, the type's lowest value, -200), and a
    long stretch whose products underflow; nothing may turn into NaN."""
    T, H = 700, 4
    ins = linear_inputs(3, (T,), H, 128, 128, dtype, "token", True, False)
    g = ins["g"]
    g[:, 0] = 0.0
    g[::50, 1] = -float("inf")
    g[10:20, 1] = torch.finfo(torch.float32).min
    g[:, 2] = -200.0
    g[:, 3] = -1.0
    out, hT = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], g, h0=ins["h0"], scale=0.1)
    check_linear(ins, (T,), out, hT, 0.1)
    g2 = torch.tensor([0.0, -float("inf"), -200.0, -1e-4], device="cuda")
    ins["g"] = g2
    out, hT = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], g2, h0=ins["h0"], scale=0.1)
    check_linear(ins, (T,), out, hT, 0.1)


def test_linear_chunk_first_token_emptied_state_forgets_h0():
    """g = -inf on the first token leaves nothing of h0: the same as no initial state, bit for bit."""
    ins = linear_inputs(5, (200,), 2, 128, 128, BF, "token", True, False)
    ins["g"][0] = -float("inf")
    a = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"])
    b = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"])
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_linear_chunk_sequences_do_not_touch(dtype):
    """NaN in one packed sequence, in the decays beside it and in the values between strided rows
    changes no bit of the others."""
    lengths = (70, 33, 200)
    ins = linear_inputs(9, lengths, 2, 128, 128, dtype, "token", True, True)
    want = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], cu_seqlens=ins["cu"])
    for name in ("q", "k", "v", "g"):
        ins[name][70:103] = float("nan")
    ins["h0"][1] = float("nan")
    torch.as_strided(ins["q"], (sum(lengths), 8), (ins["q"].stride(0), 1), 2 * 384)[:] = float("nan")
    got = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], cu_seqlens=ins["cu"])
    keep = torch.tensor([i for i in range(303) if not 70 <= i < 103], device="cuda")
    assert torch.equal(got[0][keep], want[0][keep])
    assert torch.equal(got[1][[0, 2]], want[1][[0, 2]])
    assert torch.isnan(got[0][70:103]).all() and torch.isnan(got[1][1]).all()


def test_linear_chunk_in_place_state_no_state_and_nothing():
    for T in (90, 2600):
        ins = linear_inputs(T, (T,), 2, 128, 128, BF, "token", True, False)
        out, hT = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"])
        h = ins["h0"].clone()
        out2, h2 = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=h, hT=h)
        assert h2 is h and torch.equal(out, out2) and torch.equal(hT, h)
        out3, none = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], output_final_state=False)
        assert none is None and torch.equal(out, out3)
    for dtype in (BF, FP):
        q = torch.zeros(0, 2, 64, device="cuda", dtype=dtype)
        h0 = torch.randn(1, 2, 64, 64, device="cuda")
        out, hT = kda.kda_linear_chunk_fwd(q, q, q, torch.zeros(2, device="cuda"), h0=h0)
        assert out.shape == (0, 2, 64) and torch.equal(hT, h0)
        _, hT = kda.kda_linear_chunk_fwd(q, q, q, torch.zeros(2, device="cuda"))
        assert not hT.any()
    no_device_error()


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("cu", [(0, 60, 50, 150), (0, 60, 100, 170), (0, -5, 100, 150), (3, 60, 100, 150), (0, 60, 100, 140)],
                         ids=["falling", "past-the-end", "negative", "late-start", "early-end"])
def test_linear_chunk_bad_offsets(cu, dtype):
    """Offsets that do not rise from 0 to the number of tokens set the flag and nothing is written."""
    lengths = (60, 40, 50)
    ins = linear_inputs(4, lengths, 2, 64, 64, dtype, "token", False, False)
    want = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], cu_seqlens=ins["cu"])
    no_device_error()
    out, hT = torch.full_like(want[0], 5.0), torch.full_like(want[1], 5.0)
    bad = torch.tensor(cu, dtype=torch.int32, device="cuda")
    kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], cu_seqlens=bad, out=out, hT=hT)
    assert binding.kda_get_device_error() == binding.DEVERR_BAD_SEQLENS
    assert (out == 5).all() and (hT == 5).all()
    again = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], cu_seqlens=ins["cu"])
    assert torch.equal(again[0], want[0])
    no_device_error()


# ------------------------------------------------------------------ linear attention, tokens
@pytest.mark.parametrize("N,H,dk,dv", [(1, 1, 128, 128), (1, 32, 128, 128), (3, 5, 64, 64), (7, 2, 64, 128), (6, 4, 128, 64),
                                       (65, 4, 128, 128)])
@pytest.mark.parametrize("dtype,out_dtype", [(BF, BF), (BF, FP), (FP, FP)])
@pytest.mark.parametrize("decay", ["token", "head"])
def test_linear_step(N, H, dk, dv, dtype, out_dtype, decay):
    ins = linear_inputs(N * H, (1,) * N, H, dk, dv, dtype, decay, False, True)
    r = gen(3)
    slots = 2 * N + 1
    pool = randn(r, slots, H, dk, dv)
    slot = torch.randperm(slots, generator=r, device="cuda")[:N].to(torch.int32)
    before = pool.clone()
    want, S, mag, M = linear_recurrence(f64(ins["q"]), f64(ins["k"]), f64(ins["v"]), f64(ins["g"]),
                                        h0=f64(pool[slot.long()]), cu=np.arange(N + 1), scale=0.7)
    out = kda.kda_linear_decode_step(ins["q"], ins["k"], ins["v"], ins["g"], pool, slot, scale=0.7, out_dtype=out_dtype)
    steps = 2 * F32 * 4  # the decay, its product, the sum's product and sum
    within(pool[slot.long()], S, steps * M, "state")
    inner = steps + dk * F32
    within(out, want, HALF[out_dtype] * (np.abs(want) + inner * mag) + inner * mag, "out")
    others = [i for i in range(slots) if i not in slot.tolist()]
    assert torch.equal(pool[others], before[others])
    no_device_error()


def test_linear_step_bad_slots_touch_nothing():
    ins = linear_inputs(2, (1,) * 4, 2, 128, 128, BF, "token", False, False)
    pool = torch.randn(5, 2, 128, 128, device="cuda")
    before = pool.clone()
    out = torch.full((4, 2, 128), 5.0, device="cuda", dtype=BF)
    slot = torch.tensor([4, -1, 5, 0], dtype=torch.int32, device="cuda")
    kda.kda_linear_decode_step(ins["q"], ins["k"], ins["v"], ins["g"], pool, slot, out=out)
    assert binding.kda_get_device_error() == binding.DEVERR_BAD_SLOT
    assert (out[1:3] == 5).all() and not (out[0] == 5).all() and not (out[3] == 5).all()
    assert torch.equal(pool[1:4], before[1:4])
    none = kda.kda_linear_decode_step(ins["q"][:0], ins["k"][:0], ins["v"][:0], ins["g"][:0], pool, slot[:0])
    assert none.shape == (0, 2, 128)
    no_device_error()


def test_linear_step_reset():
    """g = -inf leaves only the token itself, whatever finite state was there."""
    ins = linear_inputs(2, (1,), 1, 128, 128, FP, "token", False, False)
    pool = 1e30 * torch.randn(1, 1, 128, 128, device="cuda")
    kda.kda_linear_decode_step(ins["q"], ins["k"], ins["v"], torch.tensor([-float("inf")], device="cuda"), pool,
                               torch.zeros(1, dtype=torch.int32, device="cuda"))
    assert torch.equal(pool[0, 0], ins["k"][0, 0][:, None] * ins["v"][0, 0][None, :])


def test_prompt_then_tokens_is_one_sequence():
    """A prompt of 150 tokens and 20 single steps give what one pass over the 170 gives, within the two paths' bounds."""
    for dtype in (BF, FP):
        ins = linear_inputs(6, (170,), 2, 128, 128, dtype, "token", False, True)
        want, S, mag, M = linear_recurrence(f64(ins["q"]), f64(ins["k"]), f64(ins["v"]), f64(ins["g"]), scale=0.2)
        out, hT = kda.kda_linear_chunk_fwd(ins["q"][:150], ins["k"][:150], ins["v"][:150], ins["g"][:150], scale=0.2)
        slot = torch.zeros(1, dtype=torch.int32, device="cuda")
        outs = [out] + [kda.kda_linear_decode_step(ins["q"][t:t + 1], ins["k"][t:t + 1], ins["v"][t:t + 1], ins["g"][t:t + 1],
                                                   hT, slot, scale=0.2) for t in range(150, 170)]
        bo, bs = linear_bounds(170, 128, dtype, dtype, want, mag, M)
        within(torch.cat(outs), want, bo, "out")
        within(hT, S[:1], bs, "state")


# ------------------------------------------------------------------ streams and graphs
def test_streams_and_graphs():
    """Each operator on a side stream, and captured into a graph that is replayed on changed inputs."""
    lin = linear_inputs(8, (200,), 2, 128, 128, BF, "token", True, True)
    mm = matmul_inputs(8, 20, 384, 512)
    big = matmul_inputs(9, 300, 384, 512)
    x = randn(gen(8), 9, 512, dtype=BF)
    slot = torch.tensor([1], dtype=torch.int32, device="cuda")

    def everything(pool):
        y = kda.kda_rmsnorm_quant(x, residual=x)
        o = kda.kda_linear_chunk_fwd(lin["q"], lin["k"], lin["v"], lin["g"], h0=lin["h0"])
        t = kda.kda_linear_decode_step(lin["q"][:1], lin["k"][:1], lin["v"][:1], lin["g"][:1], pool, slot)
        return [*y, *o, t, pool, kda.kda_matmul_fp8(*mm), kda.kda_matmul_fp8(*big)]

    start = torch.randn(2, 2, 128, 128, device="cuda")
    want = everything(start.clone())
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    pool = start.clone()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = everything(pool)
    side.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    pool = start.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = everything(pool)
    for change in (False, True):
        if change:
            x.mul_(2).add_(1)
            lin["v"].mul_(0.5)
            mm[0].view(torch.uint8).fill_(0x38)  # ones
        pool.copy_(start)
        graph.replay()
        torch.cuda.synchronize()
        kept = [t.clone() for t in got]
        for a, b in zip(kept, everything(start.clone())):
            assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    no_device_error()


def test_same_call_same_bits():
    lin = linear_inputs(18, (1500, 300), 2, 128, 128, BF, "token", True, True)
    mm = matmul_inputs(19, 40, 384, 4096)
    ref = None
    for _ in range(4):
        got = [*kda.kda_linear_chunk_fwd(lin["q"], lin["k"], lin["v"], lin["g"], h0=lin["h0"], cu_seqlens=lin["cu"]),
               kda.kda_matmul_fp8(*mm)]
        assert ref is None or all(torch.equal(a, b) for a, b in zip(got, ref))
        ref = got


# ------------------------------------------------------------------ waits that run out
@pytest.mark.parametrize("what", ["matmul many rows", "matmul few rows", "linear", "linear in segments"])
def test_waits_that_run_out_are_reported_and_the_device_stays_usable(what, monkeypatch):
    """KDA_TEST_WAIT_TIMEOUT launches the variants whose waits give up at once: the call reports it, and the next
    ordinary call is right."""
    if what.startswith("matmul"):
        ins = matmul_inputs(31, *((1280, 2304, 640) if "many" in what else (5, 300, 4096)))

        def call():
            check_matmul(ins, kda.kda_matmul_fp8(*ins))
    else:
        lengths = (2500,) if "segments" in what else (300, 70)
        ins = linear_inputs(32, lengths, 2, 128, 128, BF, "token", True, False)

        def call():
            out, hT = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], cu_seqlens=ins["cu"])
            check_linear(ins, lengths, out, hT, 1.0)
    monkeypatch.setenv("KDA_TEST_WAIT_TIMEOUT", "1")
    if what.startswith("matmul"):
        kda.kda_matmul_fp8(*ins)
    else:
        kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], cu_seqlens=ins["cu"])
    assert binding.kda_get_device_error() & binding.DEVERR_WAIT_TIMEOUT
    monkeypatch.delenv("KDA_TEST_WAIT_TIMEOUT")
    for _ in range(2):
        call()
        no_device_error()


def test_waits_that_run_out_in_a_pair_of_ctas(monkeypatch):
    """The same where two CTAs share a tile and join their sums, and the same bits from call to call."""
    ins = matmul_inputs(33, 200, 4880, 2000)
    monkeypatch.setenv("KDA_TEST_WAIT_TIMEOUT", "1")
    kda.kda_matmul_fp8(*ins)
    assert binding.kda_get_device_error() & binding.DEVERR_WAIT_TIMEOUT
    monkeypatch.delenv("KDA_TEST_WAIT_TIMEOUT")
    got = [kda.kda_matmul_fp8(*ins) for _ in range(3)]
    check_matmul(ins, got[0])
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    no_device_error()


def test_segments_in_a_graph():
    """A call that runs as several kernels which may overlap, captured and replayed back to back on changed inputs."""
    lin = linear_inputs(41, (2600,), 2, 128, 128, BF, "token", True, True)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        first = kda.kda_linear_chunk_fwd(lin["q"], lin["k"], lin["v"], lin["g"], h0=lin["h0"])
        second = kda.kda_linear_chunk_fwd(lin["q"], lin["k"], lin["v"], lin["g"], h0=first[1])
    for factor in (1.0, 0.5):
        lin["v"].mul_(factor)
        graph.replay()
        graph.replay()
        torch.cuda.synchronize()
        want = kda.kda_linear_chunk_fwd(lin["q"], lin["k"], lin["v"], lin["g"], h0=lin["h0"])
        then = kda.kda_linear_chunk_fwd(lin["q"], lin["k"], lin["v"], lin["g"], h0=want[1])
        for a, b in zip((*first, *second), (*want, *then)):
            assert torch.equal(a, b)
    no_device_error()
