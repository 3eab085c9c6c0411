"""Every kernel that is launched with launch_dependent (csrc/dependent.cuh) waits for the one in front of it before anything else that it
may read or write: the wait stands in its body itself, under no condition, and in front of the first return."""
import os
import re

import pytest

from test_dependent_loads import CSRC, body, source

WAIT = re.compile(r"\b(wait_for_earlier|start_after_earlier)\(\);")
NAMES = [(f, k) for f in sorted(os.listdir(CSRC)) if f.endswith((".cu", ".cuh"))
         for k in sorted(set(re.findall(r"__global__[^;{]*?\b(\w+_kernel)\s*\(", source(f), flags=re.S))) if "earlier();" in body(source(f), k)]


def waits_at_once(text):
    """text: a kernel's definition."""
    text = text[text.index("{"):]
    for m in WAIT.finditer(text):
        front = text[:m.start()]
        if front.count("{") - front.count("}") != 1:
            continue
        line = front[max(front.rfind(c) for c in ";{}"):]          # what stands between the statement before and this one
        if re.search(r"\b(if|else|for|while)\b", line):
            continue
        returns = [r.start() for r in re.finditer(r"\breturn;", front)]
        return all(WAIT.search(front[front.rfind("{", 0, r):r]) for r in returns)
    return False


def test_the_check_tells_them_apart():
    assert waits_at_once("k(A a) { int x; start_after_earlier(); if (x) return; }")
    assert waits_at_once("k(A a) { if (odd) { wait_for_earlier(); note(); return; } wait_for_earlier(); }")
    assert not waits_at_once("k(A a) { if (odd) return; wait_for_earlier(); }")
    assert not waits_at_once("k(A a) { if constexpr (A::X) { begin(); } else { wait_for_earlier(); } }")
    assert not waits_at_once("k(A a) { read(); if (A::X) wait_for_earlier(); }")


def test_launched_kernels_are_among_them():
    launched = {k for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh"))
                for k in re.findall(r"launch_dependent\((\w+_kernel)", source(f))}
    assert {"cache4_attn_kernel", "prefix_attn_kernel", "prefix_combine_kernel"} <= launched <= {k for _, k in NAMES}


@pytest.mark.parametrize("name,kernel", NAMES)
def test_kernel_waits_at_once(name, kernel):
    assert waits_at_once(body(source(name), kernel))


def test_nothing_runs_beside_an_earlier_kernel():
    """No call starts a kernel's work before its wait."""
    for f in os.listdir(CSRC):
        if f.endswith((".cu", ".cuh")):
            assert "beside_earlier" not in source(f) and "let_follower" not in source(f), f
