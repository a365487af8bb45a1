"""Every kernel orders the initialisation of its mbarriers before their first use: one thread initialises them for the whole
CTA, so an unconditional __syncthreads() has to stand between that block and whatever waits, announces bytes or
starts a copy on one. A missing one cannot be provoked reliably, so it is looked for in the sources."""

import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "ternary_weight_only_tern_b200", "csrc")
SOURCES = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
USES = re.compile(r"grid_launch_dependents|grid_dependency_wait|mbar_wait|mbar_poll|mbar_arrive|expect|bulk|tma_load|commit\(|issue\(")


def without_comments(text):
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


def end_of_block(text, at):
    """Index behind the brace that closes the one at text[at]."""
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return i + 1
    raise AssertionError("unbalanced braces")


def unordered(text):
    """Places of one-thread blocks that initialise mbarriers and are not followed by a CTA barrier before a use."""
    text, found = without_comments(text), []
    for m in re.finditer(r"if \(threadIdx\.x == 0\) \{", text):
        end = end_of_block(text, m.end() - 1)
        if "mbar_init(" not in text[m.start():end]:
            continue
        sync = text.find("__syncthreads();", end)
        between = text[end:sync] if sync >= 0 else text[end:]
        depth = between.count("{") - between.count("}")      # 0: the barrier stands beside the block, under no condition
        if sync < 0 or depth != 0 or USES.search(re.sub(r'asm volatile\(.*?\);', "", between, flags=re.S)):
            found.append(text[:m.start()].count("\n"))
    return found


@pytest.mark.parametrize("path", SOURCES, ids=[os.path.basename(p) for p in SOURCES])
def test_a_cta_barrier_follows_the_initialisation(path):
    with open(path) as f:
        assert unordered(f.read()) == []


def test_the_search_finds_a_missing_and_a_conditional_barrier():
    init = "if (threadIdx.x == 0) {\n mbar_init(b, 1);\n fence_barrier_init();\n }\n"
    assert unordered(init + "__syncthreads();\n mbar_wait(b, 0);") == []
    assert unordered(init + "grid_dependency_wait();\n __syncthreads();") == [0]
    assert unordered(init + "if (split) {\n __syncthreads();\n }\n mbar_wait(b, 0);") == [0]
    assert unordered(init + "mbar_wait(b, 0);  // __syncthreads();") == [0]


def test_the_kernels_with_barriers_are_looked_at():
    names = set()
    for path in SOURCES:
        with open(path) as f:
            if re.search(r"if \(threadIdx\.x == 0\) \{[^}]*mbar_init\(", f.read()):
                names.add(os.path.basename(path))
    assert {"tern_decode1.cu", "tern_decodem.cu", "tern_gemm_sm100.cu", "tern_gemv.cu", "tern_nib_linear.cu",
            "tern_nib_gemm.cu", "tern_cache_attention.cu"} <= names
