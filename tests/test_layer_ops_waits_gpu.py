"""Waits of the serving operators that reach their limit: KDA_TEST_WAIT_TIMEOUT=stall launches variants with the
ordinary waits whose first CTA starts no MMA.  Nothing here traps or hangs: every wait is counted, and the time a
call may take is part of the test."""
import time

import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from gated_delta_rule_08_gb300 import binding
from layer_util import gen, linear_inputs, randn

pytestmark = pytest.mark.gpu
BF, FP8 = torch.bfloat16, torch.float8_e4m3fn

#: rows, columns, depth.  "few rows": one CTA a tile; "cluster": K over eight CTAs; "pair": two CTAs a tile
PRODUCTS = {"many rows": (1280, 2304, 640), "few rows": (5, 300, 256), "cluster": (5, 300, 4096), "pair": (200, 4880, 2000)}
SEQUENCES = {"one pass": (300, 70), "segments": (2500,)}


def product_inputs(M, N, K):
    r = gen(M + N + K)
    kb, nb = -(-K // 128), -(-N // 128)
    a, b = ((80 * randn(r, n, K)).clamp(-448, 448).to(FP8) for n in (M, N))
    return a, torch.exp(randn(r, M, kb)) / 80, b, torch.exp(randn(r, nb, kb)) / 80


def stalled(call, monkeypatch):
    """The result of a call whose first CTA stalls; a limit is a second, and a call has few of them in a row."""
    torch.cuda.synchronize()
    monkeypatch.setenv("KDA_TEST_WAIT_TIMEOUT", "stall")
    start = time.monotonic()
    got = call()
    torch.cuda.synchronize()
    took = time.monotonic() - start
    monkeypatch.delenv("KDA_TEST_WAIT_TIMEOUT")
    assert binding.kda_get_device_error() == binding.DEVERR_WAIT_TIMEOUT
    assert took < 10, took
    return got


@pytest.mark.parametrize("what", PRODUCTS)
def test_product_reports_a_wait_that_runs_out_within_seconds(what, monkeypatch):
    ins = product_inputs(*PRODUCTS[what])
    want = kda.kda_matmul_fp8(*ins)
    stalled(lambda: kda.kda_matmul_fp8(*ins), monkeypatch)
    for _ in range(2):
        assert torch.equal(kda.kda_matmul_fp8(*ins), want)
    assert binding.kda_get_device_error() == 0


@pytest.mark.parametrize("what", SEQUENCES)
def test_sequences_report_a_wait_that_runs_out_within_seconds(what, monkeypatch):
    ins = linear_inputs(32, SEQUENCES[what], 2, 128, 128, BF, "token", True, False)

    def call():
        return kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], cu_seqlens=ins["cu"])

    want = call()
    stalled(call, monkeypatch)
    for _ in range(2):
        assert all(torch.equal(a, b) for a, b in zip(call(), want))
    assert binding.kda_get_device_error() == 0


@pytest.mark.parametrize("what", ["few rows", "cluster", "pair"])
def test_product_of_a_stalled_cluster_is_not_written(what, monkeypatch):
    """The CTAs that share a tile's depth add one another's sums.  If one of them has none, the tile is left as it
    was, by all of them, and every other tile is right."""
    ins = product_inputs(*PRODUCTS[what])
    want = kda.kda_matmul_fp8(*ins)
    out = torch.full_like(want, -7.0)
    stalled(lambda: kda.kda_matmul_fp8(*ins, out=out), monkeypatch)
    rows, cols = (128, 256) if what == "pair" else (want.shape[0], 128)
    assert (out[:rows, :cols] == -7).all()
    want[:rows, :cols] = -7
    assert torch.equal(out, want)


def test_sequence_of_a_stalled_segment_is_not_written(monkeypatch):
    """A (sequence, head) of which a segment's contribution is missing keeps what was in out and hT, in all its
    segments; the other head and the other sequence are right."""
    ins = linear_inputs(33, (2500, 1400), 2, 128, 128, BF, "token", True, False)

    def call(**kw):
        return kda.kda_linear_chunk_fwd(ins["q"], ins["k"], ins["v"], ins["g"], h0=ins["h0"], cu_seqlens=ins["cu"], **kw)

    want = call()
    out, hT = torch.full_like(want[0], -7.0), torch.full_like(want[1], -7.0)
    stalled(lambda: call(out=out, hT=hT), monkeypatch)
    assert (out[:2500, 0] == -7).all() and (hT[0, 0] == -7).all()
    want[0][:2500, 0] = -7
    want[1][0, 0] = -7
    assert torch.equal(out, want[0]) and torch.equal(hT, want[1])
    assert all(not (t == -7).all() for t in call())
