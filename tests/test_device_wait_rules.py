"""Rules of the kernels' waits that a run on a GPU would show only by chance (or by a hang), read
off the sources: no GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "weight_only_bit_q4_gb300", "csrc")
KERNEL_FILES = sorted(f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")) and f != "q4_sm100.cuh")


def code(name):
    """A source without its comments (the lines stay)."""
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    text = re.sub(r"/\*.*?\*/", lambda m: "\n" * m.group(0).count("\n"), text, flags=re.S)
    return re.sub(r"//[^\n]*", "", text)


@pytest.mark.parametrize("name", KERNEL_FILES)
def test_a_lanes_own_poll_decides_nothing(name):
    """mbarrier.try_wait answers every lane apart; a branch on it that holds a warp-wide shuffle
    (warp_wait does) would name lanes that are not there.  So polls go through the bounded waits of
    q4_sm100.cuh, or the whole warp votes on them."""
    text = code(name)
    for m in re.finditer(r"\bmbar_try_wait\(", text):
        voted = text[:m.start()].rstrip().endswith("__all_sync(0xffffffffu,")
        assert voted, text[max(0, m.start() - 80):m.end() + 40]
