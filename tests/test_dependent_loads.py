"""Kernels that may start while the one in front of them still runs (csrc/dependent.cuh) read what it may have written with
ordinary loads: a non-coherent load (__ldg, ld.global.nc) is only defined for data that nothing writes during the kernel's life."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "free_block_sparse_gb300", "csrc")
NON_COHERENT = re.compile(r"__ldg\s*\(|\.global(?:\.\w+)*\.nc\b|\bld_stream_v4\s*\(|__ldlu\s*\(")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", "", f.read(), flags=re.S)


def body(text, kernel):
    """The kernel's definition, from its name to the brace that closes it."""
    at = re.search(r"\b%s\s*\([^;{]*\{" % kernel, text, flags=re.S)
    depth, i = 1, at.end()
    while depth:
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        i += 1
    return text[at.start():i]


def test_the_check_finds_such_loads():
    assert NON_COHERENT.search('x = __ldg(p + 1);') and NON_COHERENT.search('asm("ld.global.nc.L1::no_allocate.v8.b32 {")')
    assert NON_COHERENT.search('asm("ld.weak.global.nc.b32")') and not NON_COHERENT.search('asm("ld.global.L1::no_allocate.v8.b32 {")')


@pytest.mark.parametrize("name", ["cache4.cu", "cache4_attn.cu", "rowsplit.cuh", "window_attn.cu", "window_decode.cu", "window_v.cu", "norm_rope.cu"])
def test_serving_kernels_read_with_ordinary_loads(name):
    assert not NON_COHERENT.findall(source(name))


def test_the_copy_of_v_reads_with_ordinary_loads():
    assert not NON_COHERENT.findall(body(source("permute.cu"), "convert_v_f16_kernel"))


def test_every_file_with_dependent_kernels_is_looked_at():
    waits = sorted(f for f in os.listdir(CSRC) if "wait_for_earlier();" in source(f) and f != "dependent.cuh")
    assert waits == ["cache4.cu", "cache4_attn.cu", "norm_rope.cu", "permute.cu", "rowsplit.cuh", "window_attn.cu", "window_decode.cu", "window_v.cu"]
