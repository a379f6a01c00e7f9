"""Reading test of the e4m3 kernels' sources: instructions of whole warps are
reached converged, and what one lane issues is ordered behind what the others
waited for.

Tensor-memory loads and allocation, cluster barriers and named barriers are
`.aligned`: every lane has to reach them together.  After code of single lanes
(`if (lane == 0) ...`, a loop over lanes) the compiler may bring the lanes
together again by itself, but only __syncwarp() (or another instruction that
waits for all lanes) promises it.  A vote brings lanes together too but, unlike
__syncwarp(), orders no memory among them."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(__file__), "..", "w4a4_mxfp4_outlier_b200", "csrc")
FILES = ["fp8_gemm.cu", "fp8_moe.cu", "fp8_quant.cu"]

ALIGNED = re.compile(r"\b(tmem_ld_now|tmem_alloc|tmem_alloc_pair|tmem_relinquish|tmem_relinquish_pair|"
                     r"tmem_dealloc|tmem_dealloc_pair|cluster_arrive|cluster_wait|cluster_sync_all|"
                     r"named_bar_sync|named_bar_or|setmaxnreg_\w+)\s*(<[^;]*?>)?\(")
CONVERGES = re.compile(r"__syncwarp\(\)|__syncthreads\(\)|_sync\(0xFFFFFFFFu|\bwarp_wait_bounded\(|"
                       r"\bfinish_sync\(\)|\bfinish_any\(|\bmoe_last_arrival\(")
DIVERGES = re.compile(r"lane == 0\b|\btid == 0\b|\belect_one\(\)|lane >> 4|\(tid & 31\) == 0|"
                      r"\bfp8_quant_rows4\(|\bmbar_wait_bounded\(|for \([^)]*\b(tid|lane|threadIdx)\b")


def _code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    text = re.sub(r"//[^\n]*", "", text)
    # the inside of asm statements is not control flow
    return re.sub(r"asm volatile\(.*?\);", lambda m: "\n" * m.group(0).count("\n"), text, flags=re.S)


def _functions(name):
    """(first line, lines) of each function: bodies that open at the left margin."""
    lines = _code(name).split("\n")
    start = None
    for i, line in enumerate(lines):
        if start is None and line and not line[0].isspace() and line[0] not in "}#" and "namespace" not in line:
            start = i
        if start is not None and (line == "}" or (line and not line[0].isspace() and line.rstrip().endswith("}"))):
            yield start, lines[start:i + 1]
            start = None
        elif start is not None and line.startswith("};"):
            start = None


def _reached_diverged(lines):
    """Lines with an instruction of whole warps behind single lanes' code, nothing between."""
    found, diverged = [], None
    for i, line in enumerate(lines):
        events = sorted([(m.start(), "c") for m in CONVERGES.finditer(line)] +
                        [(m.start(), "d") for m in DIVERGES.finditer(line)] +
                        [(m.start(), "a") for m in ALIGNED.finditer(line)])
        for _, what in events:
            if what == "c":
                diverged = None
            elif what == "d":
                diverged = i
            elif diverged is not None and not re.match(r"\s*(template|__device__|static|if \(warp == 1\))", line):
                found.append((i, line.strip(), lines[diverged].strip()))
    return found


@pytest.mark.parametrize("name", FILES)
def test_whole_warps_are_converged(name):
    bad = []
    for first, lines in _functions(name):
        bad += [f"{name}:{first + i + 1}: {line!r} behind {why!r}" for i, line, why in _reached_diverged(lines)]
    assert not bad, "\n".join(bad)


def test_the_reading_sees_functions_and_faults():
    assert sum(1 for _ in _functions("fp8_moe.cu")) > 15 and sum(1 for _ in _functions("fp8_gemm.cu")) > 8
    text = ["void f() {", "  if (lane == 0) mbar_arrive(x);", "  tmem_ld_now(a, r);", "}"]
    assert len(_reached_diverged(text)) == 1
    assert not _reached_diverged(text[:2] + ["  __syncwarp();"] + text[2:])
    assert not _reached_diverged(text[:2] + ["  if (!warp_wait_bounded(&b, 0u, f, E)) break;"] + text[2:])


def test_copies_are_ordered_behind_every_lane_s_flags():
    # lanes acquire different flags; before one of them issues the copies a
    # __syncwarp() has to follow the vote
    lines = _code("fp8_moe.cu").split("\n")
    votes = [i for i, l in enumerate(lines) if "counter_wait_bounded(a.ready" in l]
    assert len(votes) == 1
    behind = [l for l in lines[votes[0] + 1:] if "__syncwarp()" in l or "elect_one()" in l or "fence_proxy" in l]
    assert "__syncwarp()" in behind[0], behind[0]
