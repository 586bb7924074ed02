"""Sizes at which the 32-bit numbers of the linear attention kernels would end (no GPU: refusals only)."""
import pytest

from test_layer_ops_abi import UNSUPPORTED, chunk, lib  # noqa: F401

LIMIT = 2 ** 31 - 1024


@pytest.mark.parametrize("cu", [None, 0x7000], ids=["equal", "offsets"])
@pytest.mark.parametrize("dt", [0, 1], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T", [LIMIT + 1, 2 ** 31 - 64, 2 ** 31 - 1])
def test_token_counts_whose_numbers_would_overflow_are_refused(lib, T, dt, cu):  # noqa: F811
    import ctypes
    assert chunk(lib, T=T, dt=dt, cu=None if cu is None else ctypes.c_void_p(cu)) == UNSUPPORTED
    assert lib.kda_linear_chunk_fwd_workspace_size(1, T, 2, 128, 128, dt) == 0


def test_the_furthest_token_number_fits():
    """bf16: the decays are fetched four chunks ahead of the last, partial one; fp32: two stages of eight tokens."""
    for rows in (LIMIT, LIMIT - 1, LIMIT - 63):
        last_chunk = -(-rows // 64) - 1
        assert (last_chunk + 4) * 64 + 63 < 2 ** 31
        last_stage = (rows - 1) // 8 * 8
        assert last_stage + 5 * 8 + 8 + 31 < 2 ** 31


def test_workspace_of_sizes_that_no_call_takes(lib):  # noqa: F811
    f = lib.kda_linear_chunk_fwd_workspace_size
    assert f(16385, 64, 1, 128, 128, 0) == 0 and f(16384, 64, 1 << 20, 128, 128, 0) == 0
    assert f(1, 1 << 62, 1 << 30, 128, 128, 0) == 0 and f(16384, LIMIT, 1, 64, 64, 0) > 0
