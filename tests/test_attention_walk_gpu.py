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
