"""Every kernel launch's own result is read before the next launch: a call must not report success over work that was
never started, and a later launch's success says nothing of an earlier one (no GPU)."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_08_gb300", "csrc")
LAUNCH = re.compile(r"<<<|\blaunch_after\(|\bcudaLaunchKernelEx\(")


def unchecked(text):
    """Lines of <<<>>> launches that are followed by another launch, or the function's end, before cudaGetLastError."""
    text = re.sub(r"//[^\n]*", "", text)
    found = []
    for m in re.finditer("<<<", text):
        end = text.find("\n}\n", m.end())
        rest = text[m.end():end if end >= 0 else len(text)]
        ask, other = rest.find("cudaGetLastError"), LAUNCH.search(rest)
        branch = other is not None and re.search(r"\belse\b|\breturn\b", rest[:other.start()])
        if ask < 0 or (other is not None and other.start() < ask and not branch):
            found.append(text[:m.start()].count("\n") + 1)
    return found


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu"))), ids=os.path.basename)
def test_launches_are_checked(path):
    assert unchecked(open(path).read()) == []


def test_the_search_finds_a_launch_without_a_check():
    assert unchecked("f() {\n  a<<<1, 1>>>();\n  return launch_after(b);\n}\n") == [2]
    assert unchecked("f() {\n  a<<<1, 1>>>();\n  e = launch_after(b);\n  return cudaGetLastError();\n}\n") == [2]
    assert unchecked("f() {\n  a<<<1, 1>>>();\n  if (cudaGetLastError()) return;\n  b<<<1, 1>>>();\n  return cudaGetLastError();\n}\n") == []
