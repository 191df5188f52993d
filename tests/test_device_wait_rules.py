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


@pytest.mark.parametrize("name", KERNEL_FILES)
def test_a_stage_is_released_behind_a_fence(name):
    """An arrival that lets a copy refill a stage comes from the helper that puts a fence between
    the warp's reads and the arrival.  (done_bar guards no stage: it ends the tile kernel.)"""
    for m in re.finditer(r"\bmbar_arrive\(([^;]*)\);", code(name)):
        assert m.group(1).strip() == "done_bar", m.group(0)


def test_the_release_helper_has_its_fence():
    text = code("q4_sm100.cuh")
    body = re.search(r"void warp_release\([^)]*\)\s*\{(.*?)\n\}", text, flags=re.S).group(1)
    fence, meet, arrive = (body.index(w) for w in ("__threadfence_block();", "__syncwarp();", "mbar_arrive("))
    assert fence < meet < arrive


def test_a_refill_by_the_reading_warp_is_behind_a_fence():
    """The expert kernel refills a slot from the warp that has read it, without a barrier."""
    text = code("q4_moe.cu")
    refills = [m.start() for m in re.finditer(r"if \(lane == 0 && is\.left > 0\) issue\(\);", text)]
    assert refills
    for at in refills:
        assert re.search(r"__threadfence_block\(\);\s*__syncwarp\(\);\s*$", text[:at])


@pytest.mark.parametrize("kernel,load", [("q4_moe_router_kernel", "load_w"), ("q4_moe_router_mma_kernel", "load_w")])
def test_router_weights_are_loaded_after_the_wait(kernel, load):
    """A kernel before the router may write w_router (a cast, a merge, another projection) and may
    let the router start before it is done: until griddepcontrol.wait its rows may be prefetched
    into L2, not read."""
    text = code("q4_moe.cu")
    body = text[text.index(kernel + "(const RouterParams p)"):]
    body = body[:body.index("\n}\n")]
    waits = [m.start() for m in re.finditer(r"pdl_wait_previous\(\);", body)]
    calls = [m.start() for m in re.finditer(r"(?<!auto )\b%s\(" % load, body)]
    assert calls and waits
    # the last wait is the routing CTAs' (the one before it belongs to the CTAs that prepare x)
    assert min(calls) > waits[-1]
    # (inside load_w, which is defined before the wait, stands the only other read)
    before = re.sub(r"auto %s = .*?\n  \};" % load, "", body[:waits[-1]], flags=re.S)
    assert not re.search(r"\bld_(global|nc)_\w+\(|__ldg\(", before)
