"""Paths of the serving operators' kernels that depend on sizes: more tiles of a product than CTAs, and sequences
that are cut into segments, for every head size, type, batch form and decay."""
import numpy as np
import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from gated_delta_rule_08_gb300 import binding
from layer_util import f64, linear_bounds, linear_inputs, rel2, within
from oracle.layer import linear_recurrence
from test_layer_ops_gpu import check_linear, check_matmul, matmul_inputs

pytestmark = pytest.mark.gpu
BF, FP = torch.bfloat16, torch.float32


def no_device_error():
    assert binding.kda_get_device_error() == 0


# ------------------------------------------------------------------ product: several tiles to a CTA
@pytest.mark.parametrize("M,N,K", [(2500, 4200, 16), (2500, 4200, 400), (2500, 4200, 1040), (2500, 4200, 1168), (2500, 4201, 272),
                                   (5000, 2305, 144)])
@pytest.mark.parametrize("out_dtype", [BF, FP], ids=["bf16", "fp32"])
def test_matmul_of_more_tiles_than_ctas(M, N, K, out_dtype):
    """340 and 400 tiles on 152 SMs: barriers, accumulators, scale groups and the output's staging go on from tile to
    tile, with numbers of K blocks (1 to 10) that are no multiple of the stages, of the accumulators or of a group."""
    ins = matmul_inputs(M + N + K, M, N, K)
    check_matmul(ins, kda.kda_matmul_fp8(*ins, out_dtype=out_dtype))
    no_device_error()


# ------------------------------------------------------------------ linear attention in segments
def run_and_check(ins, lengths, scale=0.1, **kw):
    out, hT = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], scale=scale, **kw)
    want, S, mag, M = linear_recurrence(f64(ins["q"]), f64(ins["k"]), f64(ins["v"]), f64(ins["g"]), h0=f64(ins["h0"]),
                                        cu=np.concatenate([[0], np.cumsum(lengths)]), scale=scale)
    bo, bs = linear_bounds(max(lengths), ins["q"].shape[2], BF, out.dtype, want, mag, M)
    within(out, want, bo, "out")
    within(hT, S, bs, "state")
    assert rel2(out, want) <= 2.0 ** -7  # three roundings to bf16 at random
    # at random: the weights of a chunk's tokens (5 steps of 2^-24), its accumulations in the tensor core (7) and two
    # roundings of the state for each of at most 40 chunks (9) come to 12; the largest decays' windows are shorter
    assert rel2(hT, S) <= 2.0 ** -20
    no_device_error()
    return out, hT


@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 128), (128, 64), (128, 128)])
@pytest.mark.parametrize("out_dtype", [BF, FP], ids=["bf16", "fp32"])
@pytest.mark.parametrize("lengths", [(2500,), (1100, 40, 0, 1300)], ids=["one", "packed"])
def test_segments_of_every_head_size_and_type(lengths, dk, dv, out_dtype):
    ins = linear_inputs(dk + dv + len(lengths), lengths, 2, dk, dv, BF, "token", True, True)
    out, _ = run_and_check(ins, lengths, cu_seqlens=ins["cu"], out_dtype=out_dtype)
    assert out.dtype == out_dtype


@pytest.mark.parametrize("dk,dv", [(64, 128), (128, 64)])
def test_segments_with_decays_that_empty_the_state(dk, dv):
    """An emptying token in some segments and in none of others, at a segment's first and last token, and constant
    decays that empty every token's state or none."""
    T, H = 2600, 4
    ins = linear_inputs(dk, (T,), H, dk, dv, BF, "token", True, False)
    g = ins["g"]
    g[700, 0] = -float("inf")
    g[1023:1026, 1] = torch.finfo(FP).min
    g[255::256, 2] = -200.0
    g[256::256, 3] = -float("inf")
    run_and_check(ins, (T,))
    ins["g"] = torch.tensor([0.0, -float("inf"), -200.0, -1e-4], device="cuda")
    run_and_check(ins, (T,))


@pytest.mark.parametrize("H,T", [(1, 1500), (40, 200), (60, 130)])
def test_equal_lengths_without_offsets(H, T):
    """B sequences of T tokens, cut and uncut, with and without the offsets that say the same."""
    lengths = (T, T, T)
    ins = linear_inputs(H + T, lengths, H, 128, 128, BF, "token", True, True)
    out, hT = run_and_check(ins, lengths, B=3)
    again = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], cu_seqlens=ins["cu"], scale=0.1)
    assert rel2(again[0], f64(out)) <= 2.0 ** -7 and rel2(again[1], f64(hT)) <= 2.0 ** -20  # cut elsewhere, perhaps


@pytest.mark.parametrize("dtype", [BF, FP], ids=["bf16", "fp32"])
def test_more_sequences_than_are_ordered(dtype):
    """Beyond 64 sequences they are taken as they come; lengths of 0, of 1 and around a chunk among them."""
    lengths = tuple([0, 1, 63, 64, 65, 7, 130, 2][i % 8] for i in range(101))
    ins = linear_inputs(101, lengths, 2, 64, 64, dtype, "token", True, False)
    out, hT = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], cu_seqlens=ins["cu"], scale=0.3)
    check_linear(ins, lengths, out, hT, 0.3)
    no_device_error()


@pytest.mark.parametrize("cu", [(0, 1800, 1700, 2500), (0, 60, 100, 2600), (0, -5, 100, 2500), (3, 60, 100, 2500), (0, 60, 100, 2400)],
                         ids=["falling", "past-the-end", "negative", "late-start", "early-end"])
def test_bad_offsets_of_sequences_in_segments(cu):
    """All three kernels of a cut call leave when the offsets are bad: nothing is written, the flag is set."""
    ins = linear_inputs(14, (1000, 700, 800), 1, 128, 64, BF, "token", True, False)
    want = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], cu_seqlens=ins["cu"])
    no_device_error()
    out, hT = torch.full_like(want[0], 5.0), torch.full_like(want[1], 5.0)
    kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], out=out, hT=hT,
                             cu_seqlens=torch.tensor(cu, dtype=torch.int32, device="cuda"))
    assert binding.kda_get_device_error() == binding.DEVERR_BAD_SEQLENS
    assert (out == 5).all() and (hT == 5).all()
    again = kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], cu_seqlens=ins["cu"])
    assert all(torch.equal(a, b) for a, b in zip(again, want))
    no_device_error()
