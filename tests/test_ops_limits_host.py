"""Limits of the quantised and backward operations that a GPU is not needed for."""
import os
import re

import pytest

import all_reduce_epilogue_gb300 as are


@pytest.fixture(scope="module")
def lib():
    from all_reduce_epilogue_gb300 import build
    build.build()
    return are.load_library()


@pytest.mark.parametrize("M,N,ok", [
    (2 ** 31 - 512, 8, True),
    (2 ** 31 - 511, 8, False),   # the tiles' tokens would pass 2^31: nothing would be launched
    (2 ** 31 - 8, 8, False),
    (1, 2 ** 31 - 512, True),
    (1, 2 ** 31 - 504, False),
    (1, 2 ** 31 - 8, False),
])
def test_sizes_next_to_31_bits(lib, M, N, ok):
    for R in (1, 8):
        assert (lib.are_supports(are.OP_GEMM_AR_QWEIGHT, R, M, N, 32) == are.OK) == ok


@pytest.mark.parametrize("source", ["norm_rows.cu", "qweight.cu"])
def test_no_non_coherent_loads_under_programmatic_launch(source):
    """These kernels may start before the kernel that writes their operands has ended; a non-coherent load wants memory
    that is read-only for the whole life of the kernel, which begins before the wait."""
    path = os.path.join(os.path.dirname(are.__file__), "csrc", source)
    code = re.sub(r"//[^\n]*", "", open(path).read())
    assert "ProgrammaticStreamSerialization" in code
    assert not re.findall(r"__ldg\b|ld\.global(?:\.\w+)*\.nc\b|__restrict__", code)
