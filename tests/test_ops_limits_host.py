"""Limits of the quantised and backward operations that a GPU is not needed for."""
import copy
import os
import pickle
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


def test_qweight_holds_what_it_checked():
    """A tensor put in place of a checked one would reach the kernel unchecked: another shape, type or device."""
    import torch
    codes, scale = torch.zeros((16, 64), dtype=torch.uint8), torch.ones((16, 1), dtype=torch.bfloat16)
    w = are.QWeight(codes, scale)
    for name, value in (("codes", codes[:8]), ("scale", scale.float()), ("zero", codes), ("group", 32), ("N", 32), ("K", 256),
                        ("_key", None), ("other", 1)):
        with pytest.raises(AttributeError):
            setattr(w, name, value)
    with pytest.raises(AttributeError):
        del w.codes
    assert w.codes.data_ptr() == codes.data_ptr() and w.zero is None and (w.N, w.K, w.group) == (16, 128, 128)
    # a tensor that changes its memory or shape afterwards takes nothing from under it
    at = codes.data_ptr()
    scale.data = torch.ones((2, 1), dtype=torch.bfloat16)
    codes.fill_(7)
    codes.data = torch.zeros((4, 4), dtype=torch.uint8)
    assert w.codes.shape == (16, 64) and w.codes.data_ptr() == at and (w.codes == 7).all() and w.scale.shape == (16, 1)
    for v in (copy.copy(w), copy.deepcopy(w), pickle.loads(pickle.dumps(w))):
        assert torch.equal(v.codes, w.codes) and torch.equal(v.scale, w.scale) and (v.N, v.K, v.group) == (16, 128, 128)


@pytest.mark.parametrize("which", ["codes", "scale", "zero"])
@pytest.mark.parametrize("both", [False, True])
def test_weights_without_memory_are_refused(which, both):
    """A storage resized to nothing has the address 0, which for zero points would mean that there are none."""
    import torch

    def make():
        t = dict(codes=torch.zeros((16, 64), dtype=torch.uint8), scale=torch.ones((16, 1), dtype=torch.bfloat16),
                 zero=torch.zeros((16, 1), dtype=torch.uint8))
        return are.QWeight(**t), t

    (a, _), (b, t) = make(), make()
    if not both:
        a = are.QWeight(a.codes, a.scale)
    out = torch.zeros((2, 16), dtype=torch.bfloat16)
    are._qweights([a, b], 2, 2, 128, out, -1)
    t[which].untyped_storage().resize_(0)
    with pytest.raises(ValueError):
        are._qweights([a, b], 2, 2, 128, out, -1)
    empty = are.QWeight(torch.empty((16, 0), dtype=torch.uint8), torch.empty((16, 0), dtype=torch.bfloat16),
                        torch.empty((16, 0), dtype=torch.uint8))
    are._qweights([empty], 1, 2, 0, out, -1)
