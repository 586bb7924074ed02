"""Hand-overs between the roles of the attention kernel for many rows, in walks whose items leave the roles little time: tiles
that are cleared one after another, items without keys.  A hand-over that is missed shows as rows not written and a wait that
has run out; every call is repeated, because roles meet in another order each time."""
import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from attention_util import Batch

pytestmark = pytest.mark.gpu


def repeats(call, want, times=20):
    for _ in range(times):
        assert torch.equal(call(), want)
    assert kda.kda_get_device_error() == 0


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("H,Hkv,window,sinks", [(64, 4, 100, 0), (64, 4, 20, 5), (64, 4, 130, 3), (20, 4, 60, 0), (32, 32, 17, 40)])
def test_items_whose_tiles_are_all_cleared(d, H, Hkv, window, sinks):
    """Two tiles an item, or three with the sinks' boxes, each with values that no row of the item sees."""
    b = Batch([0, 40, 300], [1200, 501, 700], H=H, Hkv=Hkv, d=d, window=window, sinks=sinks, seed=window)
    want = b.run()
    b.check(want)
    repeats(b.run, want)


@pytest.mark.parametrize("Hkv,N", [(1, 700), (8, 90)])
def test_requests_without_keys_in_a_walk(Hkv, N):
    """One token of each of more requests than there are SMs, 32 heads a key head: requests of length zero by themselves and
    several in a row, between short and long ones, get zeros, and the others their rows."""
    lengths = [(0, 1, 700, 0, 0, 0, 130, 3, 0, 0, 0, 0, 0, 0, 257, 40)[i * 7 % 16 if i % 100 < 60 else i % 16] for i in range(N)]
    lengths[0], lengths[-1] = 0, 500
    b = Batch([max(0, n - 1) for n in lengths], [1] * N, H=32 * Hkv, Hkv=Hkv, d=64, seed=Hkv)
    b.lengths = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    for n, length in enumerate(lengths):
        if length == 0:
            b.see[n][:] = False
    want = b.step()
    b.check(want)
    assert not want[b.lengths == 0].any()
    repeats(b.step, want)


def test_items_without_rows_in_their_second_half():
    """One token of each request, 32 heads a key head: 32 rows of 256, so that the second half only takes its turns."""
    b = Batch([(i * 37) % 200 for i in range(400)], [1] * 400, H=32, Hkv=1, d=128, window=90, sinks=3, seed=1)
    want = b.step()
    b.check(want)
    repeats(b.step, want)
