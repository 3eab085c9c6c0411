"""The files whose kernels begin with start_after_earlier() (csrc/dependent.cuh) read with ordinary loads too, as
test_dependent_loads.py asks of those that wait by themselves."""
import os

import pytest

from test_dependent_loads import CSRC, NON_COHERENT, source

FILES = sorted(f for f in os.listdir(CSRC) if "start_after_earlier();" in source(f) and f != "dependent.cuh")


def test_there_are_such_files():
    assert "cache4_bounds.cu" in FILES


@pytest.mark.parametrize("name", FILES)
def test_kernels_read_with_ordinary_loads(name):
    assert not NON_COHERENT.findall(source(name))
