"""What the sources of the kernels on 16-bit tensors have to keep to, where a run that shows the opposite could hang."""

import glob
import os
import re

import pytest

from int8_hadamard_rotated_convrot_gb300 import build as cbuild


def code_of(path):
    """The source without comments, strings and characters, its lines kept."""
    keep_lines = lambda m: "\n" * m.group().count("\n")  # noqa: E731
    return re.sub(r'//[^\n]*|/\*.*?\*/|"(?:\\.|[^"\\\n])*"', keep_lines, open(path).read(), flags=re.S)


def waits_by_lane(text):
    """Lines on which each lane of a warp decides for itself whether a wait ran out: calls of wait() that no block of one
    thread is around. (A block's condition is what stands before its brace.)"""
    lines, around, start = [], [], 0
    for at in re.finditer(r"[{};]|(?<![\w.])wait\(", text):
        if at.group() == "{":
            around.append(text[start:at.start()])
        elif at.group() == "}":
            around.pop()
        elif at.group() == "wait(":
            alone = around + [text[start:at.start()]]
            if not any("lane == 0" in head or "one_thread()" in head for head in alone):
                lines.append(text.count("\n", 0, at.start()) + 1)
            continue
        start = at.end()
    assert not around
    return lines


KERNELS = sorted(p for p in glob.glob(os.path.join(cbuild.CSRC16, "*.cu")) if "Waits wait{" in open(p).read())


def test_the_rule_itself():
    assert waits_by_lane("if (warp == 0 && lane == 0) { for (;;) { if (!wait(bar, 0)) break; } }") == []
    assert waits_by_lane("if (warp >= 4) {\n if (!wait(bar, 0)) return;\n}") == [2]
    assert waits_by_lane("if (warp >= 4) { if (lane == 0) { wait(a, 0); }\n ok = wait.together(b, 0); wait(c, 1); }") == [2]


@pytest.mark.parametrize("path", KERNELS, ids=os.path.basename)
def test_a_warp_waits_as_a_whole(path):
    """A wait that runs out sends a whole warp away, or no lane of it: what follows are instructions that all have to reach."""
    assert waits_by_lane(code_of(path)) == []


def test_all_kernels_with_waits_are_looked_at():
    assert {os.path.basename(p) for p in KERNELS} == {"attention_few.cu", "attention_forward.cu", "attention_grad_kv.cu", "attention_grad_q.cu", "gated_few.cu",
                                                      "gated_gemm.cu"}


def conditions_by_lane(text):
    """The same for the kernels on 8-bit codes, whose waits are functions: statements outside blocks of one thread that go by a
    wait's result without asking all lanes. (A result that nothing reads, and one that a vote over the block follows, is none.)"""
    lines, around, start = [], [], 0
    for at in re.finditer(r"[{};]", text):
        statement, line = text[start:at.start()], text.count("\n", 0, at.start()) + 1
        waits = re.search(r"(?<![\w.])(?:mbar_)?wait(?:_cluster)?\(", statement) and "inline" not in statement
        dropped = re.search(r"(?:^|\))\s*mbar_wait\([^;]*$", statement) and not re.search(r"(?:if|return|=)[^;]*[!=&|(]\s*mbar_wait\(", statement)
        voted = "all_lanes(" in statement or "const bool got =" in statement and re.search(r"(?:__all_sync\(0xffffffffu, |__syncthreads_and\()got\)", text[at.end():])
        if waits and not dropped and not voted and not any("lane == 0" in head or "threadIdx.x == 0" in head for head in around + [statement]):
            lines.append(line)
        if at.group() == "{":
            around.append(statement)
        elif at.group() == "}":
            around.pop()
        start = at.end()
    assert not around
    return lines


OLDER = ["block_fp8_few.cu", "block_fp8_gemm.cu", "gemm_tc.cu", "lora.cu", "pack.cu"]


@pytest.mark.parametrize("name", OLDER)
def test_a_warp_of_the_8_bit_kernels_waits_as_a_whole(name):
    assert conditions_by_lane(code_of(os.path.join(cbuild.CSRC, name))) == []
    assert conditions_by_lane("{ if (!mbar_wait(a, 0)) { } }") and conditions_by_lane("{ ok = mbar_wait(a, 0); }") and not conditions_by_lane("{ mbar_wait(a, 0); }")
