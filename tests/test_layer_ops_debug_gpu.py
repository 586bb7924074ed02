"""KDA_DEBUG_CHECKS on the serving operators."""
import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from gated_delta_rule_08_gb300 import binding
from layer_util import gen, linear_inputs, randn

pytestmark = pytest.mark.gpu


def test_two_requests_on_one_slot_are_reported(monkeypatch):
    """Distinct slots (and out-of-range ones, which their own flag reports) set nothing; a repeated slot sets
    KDA_DEVERR_PRECONDITION, in the first and last places too.  Without the switch nothing is checked."""
    n = 300
    ins = linear_inputs(1, (1,) * n, 2, 64, 64, torch.bfloat16, "head", False, False)
    pool = randn(gen(2), 2 * n, 2, 64, 64)

    def flags(slot):
        kda.kda_linear_decode_step(ins["q"], ins["k"], ins["v"], ins["g"], pool, slot)
        return binding.kda_get_device_error()

    slot = torch.randperm(2 * n, generator=gen(3), device="cuda")[:n].to(torch.int32)
    monkeypatch.setenv("KDA_DEBUG_CHECKS", "1")
    assert flags(slot) == 0
    for i, j in ((0, n - 1), (7, 8), (255, 257)):
        twice = slot.clone()
        twice[j] = twice[i]
        assert flags(twice) == binding.DEVERR_PRECONDITION
    off = slot.clone()
    off[5] = off[6] = -1
    assert flags(off) == binding.DEVERR_BAD_SLOT
    monkeypatch.delenv("KDA_DEBUG_CHECKS")
    assert flags(slot) == 0
