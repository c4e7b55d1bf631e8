"""What orders the prefill kernel's warps, read from its source: faults that no run shows for certain.  No GPU."""
import os
import re

import pytest

from paged_kv_cache_75_gb300 import build as pkg_build


def without_comments(text):
    return re.sub(r"//[^\n]*", "", re.sub(r"/\*.*?\*/", "", text, flags=re.S))


def before(text, at):
    """What every path to text[at] passes through: the text before it without the blocks that closed again."""
    out, depth = [], 0
    for c in reversed(text[:at]):
        if c == "}":
            depth += 1
        elif c == "{" and depth:
            depth -= 1
        elif depth == 0:
            out.append(c)
    return "".join(reversed(out))


@pytest.fixture(scope="module")
def kernel():
    with open(os.path.join(pkg_build.CSRC, "prefill.cu")) as f:
        text = without_comments(f.read())
    text = text[text.index("paged_prefill_tc_kernel(const __grid_constant__"):]
    return text[:text.index("PFN_cuTensorMapEncodeTiled")]


def test_the_reading_itself():
    text = "wait(); if (a) { fence(); } load();"
    assert "fence" not in before(text, text.index("load")) and "wait" in before(text, text.index("load"))
    text = "wait(); fence(); if (a) { b(); { load(); } }"
    assert "fence" in before(text, text.index("load"))


def test_tensor_memory_is_read_behind_a_fence(kernel):
    """A tcgen05.ld or .mma follows another thread's tcgen05 work only behind a tcgen05.fence::after_thread_sync that
    comes after the wait, on every path."""
    places = [m.start() for m in re.finditer(r"\b(tmem_ld\d+|mma_f16_\w+)\(", kernel)]
    assert len(places) >= 6
    for at in places:
        path = before(kernel, at)
        assert path.rfind("tc_fence_after()") > path.rfind("mbar_wait(") >= 0, kernel[at - 200:at + 60]


def test_a_warp_leaves_its_waits_together(kernel):
    """A wait's outcome can differ from lane to lane (a time limit, an abort flag set meanwhile), and the collectives
    behind it want every lane: each wait's result stays with one elected thread, is broadcast from one lane, or is a
    vote of the warp."""
    waits = [m.start() for m in re.finditer(r"\bmbar_wait\(", kernel)]
    assert len(waits) >= 8
    for at in waits:
        if "if (elect_one()) {" in before(kernel, at):
            continue
        line = kernel[kernel.rfind("\n", 0, at):kernel.index(";", at)]
        behind = kernel[kernel.index(";", at) + 1:].lstrip()
        name = re.search(r"(\w+) = [^=]*$", kernel[kernel.rfind("\n", 0, at):at])
        one = "lane == 0" in line and name and behind.startswith("%s = __shfl_sync(0xffffffffu, %s, 0)" % (2 * name.groups()))
        vote = name and behind.startswith("%s = __all_sync(0xffffffffu, %s)" % (2 * name.groups()))
        assert one or vote, line


def test_an_elected_thread_meets_no_collective(kernel):
    """What one thread runs holds nothing that waits for the rest of its warp."""
    places = [m.start() for m in re.finditer(r"(\w+_sync|__syncwarp|elect_one|bar_red_or|named_bar_\w+|uniform)\(", kernel)]
    assert len(places) >= 10
    for at in places:
        assert "if (elect_one()) {" not in before(kernel, at), kernel[at - 100:at + 60]
