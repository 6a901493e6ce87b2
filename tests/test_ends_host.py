"""Refusals of LayerNorm, the embedding and the cross entropy that need no GPU: the predicate, and the
entry points' argument checks before any device access."""
import ctypes
import os
import re
import subprocess

import pytest

import all_reduce_epilogue_gb300 as are
from tests.test_ops_host import FakeWorkspace

vp = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    from all_reduce_epilogue_gb300 import build
    build.build()
    return are.load_library()


@pytest.mark.parametrize("args,ok", [
    ((are.OP_ALLREDUCE_LAYERNORM, 8, 4096, 7168, 0), True),
    ((are.OP_ALLREDUCE_LAYERNORM, 1, 1, 32776, 0), False),
    ((are.OP_ALLREDUCE_LAYERNORM, 1, 1, 12, 0), False),
    ((are.OP_ALLREDUCE_LAYERNORM, 0, 1, 64, 0), False),
    ((are.OP_ALLREDUCE_LAYERNORM_BACKWARD, 8, 0, 16384, 0), True),
    ((are.OP_ALLREDUCE_LAYERNORM_BACKWARD, 1, 1, 16392, 0), False),
    ((are.OP_ALLREDUCE_LAYERNORM_BACKWARD, 1, -1, 64, 0), False),
    ((are.OP_GEMM_CROSS_ENTROPY, 8, 4096, 8191, 4096), True),
    ((are.OP_GEMM_CROSS_ENTROPY, 1, 0, 1, 8), True),
    ((are.OP_GEMM_CROSS_ENTROPY, 1, 1, 0, 8), False),               # an empty vocabulary
    ((are.OP_GEMM_CROSS_ENTROPY, 1, 1, 8, 0), False),
    ((are.OP_GEMM_CROSS_ENTROPY, 1, 1, 8, 12), False),              # K % 8
    ((are.OP_GEMM_CROSS_ENTROPY, 9, 1, 8, 8), False),
    ((are.OP_GEMM_CROSS_ENTROPY, 8, 1, 1 << 26, 8), False),         # 2^21 tiles of the vocabulary
    ((are.OP_GEMM_CROSS_ENTROPY, 1, 1 << 30, 1 << 18, 8), False),   # tiles past 2^30
    ((are.OP_EMBEDDING_AR, 8, 0, 32768, 1), True),
    ((are.OP_EMBEDDING_AR, 1, 1, 32776, 1), False),
    ((are.OP_EMBEDDING_AR, 1, 1, 12, 1), False),
    ((are.OP_EMBEDDING_AR, 1, 1, 64, 0), False),
    ((are.OP_EMBEDDING_AR, 8, 1, 64, 1 << 28), False),              # R * V past 31 bits
    ((are.OP_EMBEDDING_AR_BACKWARD, 8, 1 << 30, 64, (1 << 28) - 1), True),
    ((are.OP_EMBEDDING_AR_BACKWARD, 1, (1 << 30) + 1, 64, 1), False),
])
def test_supports(lib, args, ok):
    assert (lib.are_supports(*args) == are.OK) == ok


def test_null_workspace(lib):
    A, f = (vp * 2)(16, 32), ctypes.c_float(1e-6)
    assert lib.are_allreduce_layernorm(A, None, 16, None, f, 16, None, 2, 4, 64, None, None) == are.EINVAL
    assert lib.are_allreduce_layernorm_backward(A, 16, 16, f, None, 16, 16, 16, 2, 4, 64, None, None) == are.EINVAL
    assert lib.are_gemm_cross_entropy(16, A, 16, 0, 8, 16, 16, 2, 4, 8, 64, None, None) == are.EINVAL
    assert lib.are_gemm_cross_entropy_backward(16, A, 16, 0, 8, 16, 16, 16, A, 2, 4, 8, 64, None, None) == are.EINVAL
    assert lib.are_embedding_ar(16, 0, A, f, 16, 2, 4, 64, 8, None, None) == are.EINVAL
    assert lib.are_embedding_ar_backward(16, 0, 16, f, 0, A, 2, 4, 64, 8, None, None) == are.EINVAL


def test_binding_refuses_host_tensors(lib):
    import torch
    ws = FakeWorkspace()
    x, g = torch.zeros((2, 64), dtype=torch.bfloat16), torch.ones(64)
    with pytest.raises(ValueError):
        are.allreduce_layernorm([x], None, g, g, 1e-6, x, ws)
    with pytest.raises(ValueError):
        are.allreduce_layernorm_backward([x], x, g, 1e-6, x, g, g, ws)
    ids, f = torch.zeros(2, dtype=torch.int64), torch.zeros(2)
    with pytest.raises(ValueError):
        are.gemm_cross_entropy(x, [x], ids, f, f, ws)
    with pytest.raises(ValueError):
        are.gemm_cross_entropy_backward(x, [x], ids, f, f, x, [x], ws)
    with pytest.raises(ValueError):
        are.embedding_ar(ids, [x], x, ws)
    with pytest.raises(ValueError):
        are.embedding_ar_backward(ids, x, [x], ws)


@pytest.mark.parametrize("source", ["rows.cuh", "layernorm.cu", "embedding.cu"])
def test_no_non_coherent_loads_under_programmatic_launch(source):
    """These kernels may start before the kernel that writes their operands has ended; a non-coherent load wants memory
    that is read-only for the whole life of the kernel, which begins before the wait."""
    code = re.sub(r"//[^\n]*", "", open(os.path.join(os.path.dirname(are.__file__), "csrc", source)).read())
    assert "launch_dependent(" in code
    assert not re.findall(r"__ldg\b|ld\.global(?:\.\w+)*\.nc\b|__restrict__", code)


SIZES_PROGRAM = r"""
#include <cstdio>
#include <cstdlib>

#include "xent_sizes.h"

int main(int argc, char** argv) {
    for (int i = 1; i + 2 < argc; i += 3) {
        are::XentSizes z{};
        const bool ok = are::xent_sizes(atoll(argv[i]), atoll(argv[i + 1]), atoll(argv[i + 2]), z);
        printf("%d %zu %zu %zu %zu\n", ok, z.sums_at(), z.h_at(), z.rows_at(), z.total());
    }
}
"""


def _sizes(tmp_path, caps):
    src, exe = tmp_path / "sizes.cpp", tmp_path / "sizes"
    src.write_text(SIZES_PROGRAM)
    csrc = os.path.join(os.path.dirname(are.__file__), "csrc")
    subprocess.run([os.environ.get("CXX", "g++"), "-std=c++17", "-I", csrc, str(src), "-o", str(exe)], check=True)
    lines = subprocess.run([str(exe), *[str(v) for c in caps for v in c]], check=True, capture_output=True, text=True).stdout
    return [[int(v) for v in line.split()] for line in lines.splitlines()]


def test_cross_entropy_buffers(tmp_path):
    """The cross entropy's buffers begin on 256 bytes and hold what a call of the capacities needs, whatever M_max and K_max
    are (workspaces take any K_max; calls have K % 8 == 0)."""
    caps = [(m, k, v) for m in (1, 2, 3, 5, 77, 129, 4096) for k in (1, 2, 7, 8, 1000, 1001, 1002, 1004, 4096)
            for v in (1, 256, 257, 8192)]
    for (m, k, v), (ok, sums, h, rows, total) in zip(caps, _sizes(tmp_path, caps), strict=True):
        assert ok and not sums % 256 and not h % 256 and not rows % 256, (m, k, v)
        assert sums >= 2 * m * -(-v // 256) * 256 * 2 and h - sums >= m * k * 4 and rows - h >= m * k * 2 and total - rows >= m * 12
    # capacities whose products pass 64 bits are refused, not wrapped
    for ok, *_ in _sizes(tmp_path, [(1, (1 << 63) - 8, 256), (1 << 62, 8, 256), (1 << 31, 1 << 31, 1), (1 << 40, 8, 1 << 28)]):
        assert not ok


def test_setters_refuse_null_workspaces(lib):
    assert lib.are_workspace_set_vocab_piece(None, 256) == are.EINVAL
    assert lib.are_workspace_set_logit_gradient(None, 2) == are.EINVAL


@pytest.mark.parametrize("source", ["cross_entropy.cu", "ptx.cuh", "norm_rows.cu", "qweight.cu"])
def test_no_non_coherent_loads_in_the_other_kernels_under_programmatic_launch(source):
    """The same of the cross entropy, of the wrappers that all of them load through, and of the earlier kernels."""
    code = re.sub(r"//[^\n]*", "", open(os.path.join(os.path.dirname(are.__file__), "csrc", source)).read())
    assert not re.findall(r"__ldg\b|ld\.global(?:\.\w+)*\.nc\b|__restrict__", code)
    if source == "ptx.cuh":
        assert re.findall(r"ld_stream_v4", code)
