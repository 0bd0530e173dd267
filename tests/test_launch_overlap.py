"""Kernels here may start while the one before them still runs (programmatic dependent launch), and wait for it before they
touch what it writes.  A read through the read-only path (__ldg, ld.global.nc, or what the compiler makes of a `const
__restrict__` parameter) is defined only for memory that nobody writes while the reading kernel runs, from its start on,
and is not held back by the wait: the kernels read global memory with ordinary loads."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "quantized_gemm_dequant_gb300", "csrc")
FILES = sorted(os.path.join(d, f) for d, _, fs in os.walk(CSRC) for f in fs if f.endswith((".cu", ".cuh")))


def _code(path):
    """The source without its comments."""
    s = re.sub(r"/\*.*?\*/", " ", open(path).read(), flags=re.S)
    return re.sub(r"//[^\n]*", "", s)


def test_sources_are_found():
    assert len(FILES) > 20 and any("pdl_wait();" in _code(f) for f in FILES)


@pytest.mark.parametrize("path", FILES, ids=[os.path.relpath(f, CSRC) for f in FILES])
def test_no_read_only_loads(path):
    s = _code(path)
    if "pdl_wait()" not in s:
        return
    assert "__ldg(" not in s and "ld.global.nc" not in s
    assert not re.search(r"\bconst\s+\w+\s*\*\s*(const\s+)?__restrict__", s)
