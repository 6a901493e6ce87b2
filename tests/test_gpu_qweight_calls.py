"""Calls of the 4-bit linear in several parts and captured ones, every output looked at."""
import pytest
import torch

import all_reduce_epilogue_gb300 as are
from tests import ops_ref as ref
from tests.gpu_util import need_gpu
from tests.test_gpu_qweight import tiled, tokens8, weights  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def test_every_replay_in_every_tile(tiled):  # noqa: F811
    """The operands of call after call written just before it, captured: the outputs of each replay, of other operands each
    time, in a staging buffer that the replay before left full."""
    ws, _ = tiled
    R, M, N, K = 4, 40, 264, 544
    made = [weights(R, N, K, 32, i % 2 == 0, 400 + i) for i in range(3)]
    sets = [m[0] for m in made]
    tokens = [[torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)] for _, g in made]
    sets = [[(c, s, torch.full_like(c[:, :17], 8) if z is None else z) for c, s, z in w] for w in sets]
    w = [tuple(torch.zeros_like(t) for t in r) for r in sets[0]]
    qw, x = [are.QWeight(*t, 32) for t in w], [torch.zeros_like(t) for t in tokens[0]]
    src = [tuple(torch.zeros_like(t) for t in r) for r in sets[0]], [torch.zeros_like(t) for t in x]
    outs = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(2)]

    def step():
        for i, out in enumerate(outs):
            for r in range(R):
                for to, of in zip(w[r], src[0][r]):
                    to.copy_(of)
                x[(r + i) % R].copy_(src[1][r])  # the ranks' tokens change places in the second call
            are.gemm_ar_qweight(x, qw, out, ws)

    step()
    torch.cuda.synchronize()
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        step()
    for i in (0, 1, 2, 1):
        for r in range(R):
            for to, of in zip(src[0][r], sets[i][r]):
                to.copy_(of)
            src[1][r].copy_(tokens[i][r])
        for o in outs:
            o.fill_(9.0)
        gr.replay()
        torch.cuda.synchronize()
        assert ws.device_status()["code"] == 0
        for j, o in enumerate(outs):
            want, tol = ref.linear64([tokens[i][(r - j) % R] for r in range(R)], sets[i], 32)
            ref.check(o, want, tol, f"operands {i}, call {j}")


@pytest.mark.parametrize("kind", ["bf16", "fp32", "e8m0"])
@pytest.mark.parametrize("R,M,N,K", [(2, 300, 72, 8192), (1, 130, 136, 10016), (2, 75, 40, 20000)])
def test_parts_into_several_views(kind, R, M, N, K):
    """More tokens than the staging buffer holds, of each kind, into a view a rank, whose last row stays."""
    need_gpu()
    w, g = weights(R, N, K, 128, True, 410 + M)
    x = [torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)]
    views = [torch.full((M + 1, N), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(R)]
    qw, out = [are.QWeight(*t, 128) for t in w], [v[:M] for v in views]
    with are.Workspace(R_max=R, M_max=1, N_max=8) as ws:
        if kind == "bf16":
            are.gemm_ar_qweight(x, qw, out, ws)
            vals = x
        else:
            t = [tokens8(v.float(), 64, kind == "e8m0") for v in x]
            are.gemm_ar_qweight_qx([v[0] for v in t], [v[1] for v in t], qw, out, ws, xgroup=64)
            vals = [v[2] for v in t]
        assert ws.device_status()["code"] == 0
    want, tol = ref.linear64(vals, w, 128)
    for v in views:
        ref.check(v[:M], want, tol, "out")
        assert (v[M] == 5).all()


def test_eight_bit_types_and_bytes_give_the_same():
    """float8_e4m3fn and float8_e8m0fnu tensors, written by the norm and read by the linear, and bytes."""
    need_gpu()
    R, M, N, K = 2, 12, 72, 320
    w, g = weights(R, N, K, 64, False, 430)
    qw = [are.QWeight(*t, 64) for t in w]
    parts = [torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)]
    gamma = torch.rand(K, generator=g, device="cuda") + 0.5
    outs = []
    with are.Workspace(R_max=R, M_max=1, N_max=K) as ws:
        for codes, scales in ((torch.uint8, torch.uint8), (torch.float8_e4m3fn, torch.float8_e8m0fnu)):
            q = torch.empty((M, K), dtype=codes, device="cuda")
            s = torch.empty((M, 10), dtype=scales, device="cuda")
            out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
            are.allreduce_rmsnorm_quant_groups(parts, None, gamma, 1e-6, q, s, ws, group=32)
            are.gemm_ar_qweight_qx((q,) * R, (s,) * R, qw, (out,) * R, ws, xgroup=32)
            outs.append((q.view(torch.uint8), s.view(torch.uint8), out))
        assert ws.device_status()["code"] == 0
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    val = outs[0][0].view(torch.float8_e4m3fn).double() * ref.e8m0_value(outs[0][1]).repeat_interleave(32, -1)
    want, tol = ref.linear64([val] * R, w, 64)
    ref.check(outs[0][2], want, tol, "out")
