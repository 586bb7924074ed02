"""The marshalling module lets other Python threads run while a C entry point does: a launch that waits (for a place in the
device's queue, or for work that needs the interpreter) must not hold the interpreter lock."""
import ctypes
import subprocess
import threading
import time

import pytest
import torch

import gated_delta_rule_08_gb300 as kda
from attention_util import BF, ints
from gated_delta_rule_08_gb300 import binding

pytestmark = pytest.mark.gpu

SOURCE = """
#include <time.h>
volatile int entered, go, seen;
int entry(void) {  /* waits for `go` for at most two seconds, as a full queue would */
  struct timespec ms = {0, 1000000};
  entered = 1;
  for (int i = 0; i < 2000 && !go; ++i) nanosleep(&ms, 0);
  seen = go;
  return 0;
}
"""


@pytest.fixture(scope="module")
def waiting(tmp_path_factory):
    """The marshalling module bound to entry points that wait, until the tests are over."""
    at = tmp_path_factory.mktemp("entry")
    (at / "entry.c").write_text(SOURCE)
    subprocess.run(["gcc", "-O1", "-shared", "-fPIC", "-o", str(at / "entry.so"), str(at / "entry.c")], check=True)
    lib = ctypes.CDLL(str(at / "entry.so"))
    module = binding._load_marshal()
    names = ("kda_block_tables", "kda_rope_append", "kda_window_attention_fwd", "kda_window_attention_decode_step", "kda_tree_attention")
    module.bind({n: ctypes.cast(lib.entry, ctypes.c_void_p).value for n in names}, binding.KdaError)
    yield lib
    binding._load_marshal()


def calls():
    q, k = torch.zeros(2, 2, 64, device="cuda", dtype=BF), torch.zeros(2, 1, 64, device="cuda", dtype=BF)
    cache, table, two = torch.zeros(4, 16, 1, 64, device="cuda", dtype=BF), ints([[0], [1]]), ints([1, 1])
    cu, mask = ints([0, 1, 2]), torch.ones(2, 1, device="cuda", dtype=torch.int64)
    freq = torch.ones(32, device="cuda", dtype=torch.float64)
    return {
        "block_tables": lambda: kda.kda_block_tables(two, two, table, ints([2, 3]), two, block_size=16, max_tokens=2),
        "rope_append": lambda: kda.kda_rope_append(q, k, k, freq, two, two, cache, cache.clone()),
        "fwd": lambda: kda.kda_window_attention_fwd(q, cache, cache, table, two, cu),
        "step": lambda: kda.kda_window_attention_decode_step(q, cache, cache, table, two),
        "tree": lambda: kda.kda_tree_attention(q, cache, cache, table, two, cu, mask),
    }


@pytest.mark.parametrize("name", ["block_tables", "rope_append", "fwd", "step", "tree"])
def test_another_thread_runs_during_a_call(waiting, name):
    entered, go, seen = (ctypes.c_int.in_dll(waiting, n) for n in ("entered", "go", "seen"))
    call = calls()[name]
    entered.value = go.value = seen.value = 0

    def other():
        end = time.monotonic() + 4
        while not entered.value and time.monotonic() < end:
            time.sleep(0.001)
        go.value = 1

    thread = threading.Thread(target=other)
    thread.start()
    call()
    thread.join()
    assert seen.value == 1, "the call held the interpreter until it gave up"
