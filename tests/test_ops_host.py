"""Refusals of the quantised and backward operations that need no GPU: the
predicate, and the C entry points' argument checks before any device access."""
import ctypes

import pytest

import all_reduce_epilogue_gb300 as are

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from all_reduce_epilogue_gb300 import build
    build.build()
    return are.load_library()


@pytest.mark.parametrize("args,ok", [
    ((are.OP_ALLREDUCE_RMSNORM_BACKWARD, 8, 4096, 7168, 0), True),
    ((are.OP_ALLREDUCE_RMSNORM_BACKWARD, 1, 0, 16384, 0), True),
    ((are.OP_ALLREDUCE_RMSNORM_BACKWARD, 1, 1, 16392, 0), False),  # N too large
    ((are.OP_ALLREDUCE_RMSNORM_BACKWARD, 1, 1, 20, 0), False),     # N % 8
    ((are.OP_ALLREDUCE_RMSNORM_BACKWARD, 9, 1, 64, 0), False),
    ((are.OP_GEMM_AR_QWEIGHT, 8, 1, 7168, 2048), True),
    ((are.OP_GEMM_AR_QWEIGHT, 1, 0, 8, 0), True),
    ((are.OP_GEMM_AR_QWEIGHT, 1, 1, 8, 48), False),                # K % 32
    ((are.OP_GEMM_AR_QWEIGHT, 1, 1, 12, 64), False),               # N % 8
    ((are.OP_GEMM_AR_QWEIGHT, 0, 1, 8, 64), False),
    ((are.OP_GEMM_AR_QWEIGHT, 1, 1 << 30, 1 << 20, 64), False),    # more CTAs than a grid holds
    ((are.OP_GEMM_AR_QWEIGHT, 1, -1, 8, 64), False),
    ((are.OP_GEMM_AR_QWEIGHT, 1, 1, 8, 1 << 20), True),
    ((are.OP_GEMM_AR_QWEIGHT, 1, 1, 8, (1 << 20) + 32), False),    # K too large
])
def test_supports(lib, args, ok):
    assert (lib.are_supports(*args) == are.OK) == ok


def test_null_workspace(lib):
    A, f = (vp * 6)(*[16] * 6), ctypes.c_float(1e-6)
    assert lib.are_allreduce_rmsnorm_quant_groups(A, None, 16, f, 0, 128, 16, 16, None, 2, 4, 64, None, None) == are.EINVAL
    assert lib.are_allreduce_rmsnorm_backward(A, 16, 16, f, None, 16, 16, 2, 4, 64, None, None) == are.EINVAL
    assert lib.are_gemm_ar_qweight(A, A, 128, A, 2, 4, 64, 64, None, None) == are.EINVAL
    assert lib.are_gemm_ar_qweight_qx(A, A, 0, 128, A, 128, A, 2, 4, 64, 64, None, None) == are.EINVAL


class FakeWorkspace:
    """As much of a workspace as the binding's checks see: they refuse before any use of the handle."""
    device_index = 0

    @property
    def handle(self):
        raise AssertionError("a refused call reached the library")


def test_binding_refuses_host_tensors(lib):
    import torch
    ws = FakeWorkspace()
    x = torch.zeros((2, 64), dtype=torch.bfloat16)
    g = torch.ones(64)
    with pytest.raises(ValueError):
        are.allreduce_rmsnorm_quant_groups([x], None, g, 1e-6, x, x, ws)
    with pytest.raises(ValueError):
        are.allreduce_rmsnorm_backward([x], x, g, 1e-6, x, g, ws)
    w = are.QWeight(torch.zeros((64, 32), dtype=torch.uint8), torch.ones((64, 1), dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        are.gemm_ar_qweight([x], [w], x, ws)
    with pytest.raises(ValueError):
        are.gemm_ar_qweight_qx([x], [x], [w], x, ws)
    with pytest.raises(ValueError):
        are.gemm_ar_qweight([], [w], x, ws)


def test_qweight_shapes():
    import torch
    c = torch.zeros((16, 80), dtype=torch.uint8)   # K = 160
    s = torch.ones((16, 2), dtype=torch.bfloat16)
    w = are.QWeight(c, s, group=128)
    assert (w.N, w.K, w.group) == (16, 160, 128)
    are.QWeight(c, torch.ones((16, 5), dtype=torch.bfloat16), torch.zeros((16, 5), dtype=torch.uint8), 32)
    for a in ((c, s, None, 32), (c, s, None, 100), (c, s.float()), (c.view(-1), s), (c.t(), s), (c, s, s)):
        with pytest.raises(ValueError):
            are.QWeight(*a)
