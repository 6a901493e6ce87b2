"""What a workspace costs those who call none of the quantised and backward operations, and their first call."""
import subprocess
import sys
import textwrap
import os

import pytest
import torch

import all_reduce_epilogue_gb300 as are
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_memory_of_narrow_workspaces():
    """2 MiB a rank of staged tokens, and scratch by N_max: sixteen workspaces for rows of 8 to 64 columns."""
    need_gpu()
    held = [are.Workspace(1, 1, 8)]  # what the first one loads
    torch.cuda.synchronize()
    free = torch.cuda.mem_get_info()[0]
    held += [are.Workspace(1, 1, 8 << i % 4) for i in range(16)]
    used = free - torch.cuda.mem_get_info()[0]
    for w in held:
        w.close()
    assert used <= 16 * (4 << 20), used


def test_first_calls_captured():
    """In a fresh process, the first call of each operation on a workspace is made inside a capture."""
    need_gpu()
    code = textwrap.dedent("""
        import sys
        import torch
        sys.path.insert(0, ROOT)
        import all_reduce_epilogue_gb300 as are
        bf = dict(dtype=torch.bfloat16, device="cuda")
        x, h, dh = (torch.full((20, 256), 2.0, **bf) for _ in range(3))
        gamma, dgamma = torch.ones(256, device="cuda"), torch.zeros(256, device="cuda")
        q, s = torch.zeros((20, 256), dtype=torch.uint8, device="cuda"), torch.zeros((20, 2), device="cuda")
        w = are.QWeight(torch.full((64, 128), 0x99, dtype=torch.uint8, device="cuda"), torch.ones((64, 2), **bf))
        out, out8 = torch.zeros((20, 64), **bf), torch.zeros((20, 64), **bf)
        spaces = [are.Workspace(1, 20, 256) for _ in range(4)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            are.allreduce_rmsnorm_quant_groups([x], None, gamma, 1e-6, q, s, spaces[0])
            are.allreduce_rmsnorm_backward([x], h, gamma, 1e-6, dh, dgamma, spaces[1])
            are.gemm_ar_qweight([x], [w], out, spaces[2])
            are.gemm_ar_qweight_qx([q], [s], [w], out8, spaces[3])
        graph.replay()
        torch.cuda.synchronize()
        for ws in spaces:
            assert ws.device_status()["code"] == 0
        # rows of 2: y = 1 / sqrt(1 + eps / 4), code 448; dy = h: dh = 0 but for eps; dgamma = 20 * 2
        assert bool((q == 0x7E).all()) and bool(((s - 1 / 448).abs() < 1e-8).all())
        assert bool((dh.abs() < 1e-5).all()) and bool(((dgamma - 40).abs() < 1e-3).all())
        assert bool((out == 512).all()) and bool((out8 == 256).all())
        print("ok")
    """).replace("ROOT", repr(ROOT))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr
