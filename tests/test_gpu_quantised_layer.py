"""The operators as a layer runs them: the norm writes 8-bit tokens, 4-bit
products read them, the ranks' sum goes through the next norm; and a training
step's forward and backward.  Each step is compared with the 64-bit result for
the tensors that went into it."""
import pytest
import torch

import all_reduce_epilogue_gb300 as are
from tests import ops_ref as ref
from tests.gpu_util import need_gpu
from tests.test_gpu_qweight import weights

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,pow2,group", [(1, False, 128), (5, True, 32), (19, False, 64)])
@pytest.mark.parametrize("graph", [False, True])
def test_decode_layer(M, pow2, group, graph):
    """norm -> column-parallel product on each rank -> row-parallel product -> norm, on one stream or captured."""
    need_gpu()
    R, N, F = 4, 1024, 512
    up, g = weights(R, F, N, 128, True, 1)
    down, _ = weights(R, N, F, 64, False, 2)
    up_q, down_q = [are.QWeight(*t, 128) for t in up], [are.QWeight(*t, 64) for t in down]
    bf = dict(dtype=torch.bfloat16, device="cuda")
    parts = [torch.empty((M, N), **bf) for _ in range(R)]
    res, res2, res3 = (torch.empty((M, N), **bf) for _ in range(3))
    gamma = 1 + 0.1 * torch.randn(N, generator=g, device="cuda")
    sdt = torch.uint8 if pow2 else torch.float32
    q = [torch.empty((M, N), dtype=torch.uint8, device="cuda") for _ in range(2)]
    s = [torch.empty((M, N // group), dtype=sdt, device="cuda") for _ in range(2)]
    mid = [torch.empty((M, F), **bf) for _ in range(R)]
    out = torch.empty((M, N), **bf)
    with are.Workspace(R_max=R, M_max=M, N_max=N) as ws:
        def layer():
            are.allreduce_rmsnorm_quant_groups(parts, res, gamma, ref.EPS, q[0], s[0], ws, group=group, residual_out=res2)
            for r in range(R):
                are.gemm_ar_qweight_qx([q[0]], [s[0]], [up_q[r]], mid[r], ws, xgroup=group)
            are.gemm_ar_qweight(mid, down_q, out, ws)
            are.allreduce_rmsnorm_quant_groups([out], res2, gamma, ref.EPS, q[1], s[1], ws, group=group, residual_out=res3)
        run = layer
        if graph:
            layer()
            cg = torch.cuda.CUDAGraph()
            with torch.cuda.graph(cg):
                layer()
            run = cg.replay
        for _ in range(3):
            for t in parts + [res]:
                t.normal_(generator=g)
            run()
            assert ws.device_status()["code"] == 0
            _, _, y, tol = ref.norm64(parts, res, gamma)
            ref.check_quant(q[0], s[0], y, tol, group, pow2)
            f = ref.e8m0_value(s[0]) if pow2 else s[0].double()
            x = q[0].view(torch.float8_e4m3fn).double() * f.repeat_interleave(group, -1)
            for r in range(R):
                want, tol = ref.linear64([x], [up[r]], 128)
                ref.check(mid[r], want, tol, f"up {r}")
            want, tol = ref.linear64(mid, down, 64)
            ref.check(out, want, tol, "down")
            _, _, y, tol = ref.norm64([out], res2, gamma)
            ref.check_quant(q[1], s[1], y, tol, group, pow2)


def test_training_step():
    """Forward through the all-reduced norm, backward through it, against autograd in 64 bits."""
    need_gpu()
    R, M, N = 4, 70, 520
    g = torch.Generator(device="cuda").manual_seed(3)
    parts = [torch.randn((M, N), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)]
    res = torch.randn((M, N), generator=g, device="cuda").to(torch.bfloat16)
    gamma = 1 + 0.1 * torch.randn(N, generator=g, device="cuda")
    out, h, dh = (torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    dgamma = torch.empty(N, device="cuda")
    dy = [(0.1 * torch.randn((M, N), generator=g, device="cuda")).to(torch.bfloat16) for _ in range(R)]
    dres = (0.1 * torch.randn((M, N), generator=g, device="cuda")).to(torch.bfloat16)
    with are.Workspace(R_max=R, M_max=M, N_max=N) as ws:
        are.allreduce_add_rmsnorm(parts, res, gamma, ref.EPS, out, h, ws)
        are.allreduce_rmsnorm_backward(dy, h, gamma, ref.EPS, dh, dgamma, ws, dres=dres)
        assert ws.device_status()["code"] == 0
    x = h.double().requires_grad_()
    gm = gamma.double().requires_grad_()
    y = x / torch.sqrt((x * x).mean(1, keepdim=True) + ref.EPS) * gm
    ((sum(t.double() for t in dy) * y).sum() + (dres.double() * x).sum()).backward()
    _, tol, _, tol_g = ref.backward64(dy, h, gamma, dres)
    ref.check(dh, x.grad, tol, "dh")
    ref.check(dgamma, gm.grad, tol_g, "dgamma")


def test_two_streams_with_a_workspace_each():
    """The same calls at once on two streams, each with its own workspace and tensors: the bits of either alone."""
    need_gpu()
    R, M, N, K = 4, 24, 512, 1024
    sides = []
    for i in range(2):
        g = torch.Generator(device="cuda").manual_seed(200 + i)
        rand = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
        parts, gamma = [rand(M, K) for _ in range(R)], torch.rand(K, generator=g, device="cuda") + 0.5
        w = [are.QWeight(torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8),
                         rand(N, K // 128) * 0.01, None, 128) for _ in range(R)]
        out = [torch.empty((M, K), dtype=torch.uint8, device="cuda"), torch.empty((M, K // 128), device="cuda"),
               torch.empty((M, N), dtype=torch.bfloat16, device="cuda"), torch.empty((M, K), dtype=torch.bfloat16, device="cuda"),
               torch.empty(K, device="cuda")]
        ws = are.Workspace(R_max=R, M_max=1, N_max=K)
        ws.set_debug(are.DEBUG_QWEIGHT_STAGED, 16 * (i + 1))
        sides.append((parts, gamma, w, out, ws, torch.cuda.Stream()))

    def step(side, stream=None):
        parts, gamma, w, (q, f, y, dh, dg), ws, _ = side
        are.allreduce_rmsnorm_quant_groups(parts, None, gamma, 1e-6, q, f, ws, group=128, stream=stream)
        are.gemm_ar_qweight_qx([q] * R, [f] * R, w, y, ws, xgroup=128, stream=stream)
        are.allreduce_rmsnorm_backward(parts, parts[0], gamma, 1e-6, dh, dg, ws, stream=stream)

    try:
        want = []
        for side in sides:
            step(side)
            torch.cuda.synchronize()
            want.append([t.clone() for t in side[3]])
            for t in side[3]:
                t.zero_()
        torch.cuda.synchronize()
        for _ in range(50):
            for side in sides:
                step(side, side[5])
        torch.cuda.synchronize()
        for side, expected in zip(sides, want):
            assert side[4].device_status()["code"] == 0
            for t, e in zip(side[3], expected):
                assert torch.equal(t, e)
    finally:
        for side in sides:
            side[4].close()
