"""Backward pass of all-reduce + residual + RMSNorm."""
import pytest
import torch

import all_reduce_epilogue_gb300 as are
from tests import ops_ref as ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    need_gpu()
    with are.Workspace(R_max=8, M_max=1, N_max=16384) as w:
        yield w


def inputs(R, M, N, seed, dres=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    dy = [(r(M, N) * 0.01).to(torch.bfloat16) for _ in range(R)]
    return dy, (r(M, N) * 3).to(torch.bfloat16), 1 + 0.1 * r(N), (r(M, N) * 0.01).to(torch.bfloat16) if dres else None


def run(ws, dy, h, gamma, dres, dgamma=True, dh=None):
    M, N = h.shape
    dh = torch.empty((M, N), dtype=torch.bfloat16, device="cuda") if dh is None else dh
    dg = torch.full((N,), 7.0, device="cuda") if dgamma else None
    are.allreduce_rmsnorm_backward(dy, h, gamma, ref.EPS, dh, dg, ws, dres=dres)
    assert ws.device_status()["code"] == 0
    return dh, dg


# one row (one block: its sums are dgamma), a block a row, several rows a block, each packs-per-thread variant
@pytest.mark.parametrize("R,M,N,dres", [(1, 1, 8, True), (8, 1, 7168, True), (2, 2, 40, False), (3, 7, 264, True),
                                        (1, 151, 1024, True), (1, 1000, 2048, False), (5, 305, 2056, True),
                                        (4, 33, 4096, False), (8, 620, 4104, True), (3, 9, 5000, True), (8, 311, 7168, True),
                                        (8, 2, 8192, False), (2, 160, 8200, True), (8, 157, 16384, True), (1, 2500, 64, True),
                                        (1, 400, 7680, True), (3, 200, 7688, False), (4, 170, 11528, True), (1, 160, 15368, True)])
def test_against_64_bits(ws, R, M, N, dres):
    dy, h, gamma, e = inputs(R, M, N, 100 * R + M + N, dres)
    if M > 4:
        h[3] = 0              # a padded row: inv = eps^-1/2
        for t in dy:
            t[2] = 0
    dh, dg = run(ws, dy, h, gamma, e)
    want, tol, want_g, tol_g = ref.backward64(dy, h, gamma, e)
    ref.check(dh, want, tol, "dh")
    ref.check(dg, want_g, tol_g, "dgamma")
    again = run(ws, dy, h, gamma, e)
    assert torch.equal(again[0], dh) and torch.equal(again[1], dg)
    # a frozen gamma and an in-place residual gradient give the same bits
    into = e.clone() if dres else None
    dh2, none = run(ws, dy, h, gamma, into, dgamma=False, dh=into)
    assert none is None and torch.equal(dh2, dh)
    assert ws.last_launch()["kernel"] == "norm_backward_rows_kernel"


def test_against_differences(ws):
    """The gradient of L = sum(dy * y) + sum(dres * h) by central differences of the forward formula in 64 bits."""
    dy, h, gamma, e = inputs(3, 4, 96, 77)
    dh, dg = run(ws, dy, h, gamma, e)
    d, x, gm = sum(t.double() for t in dy), h.double(), gamma.double()

    def loss(x, gm):
        y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + ref.EPS) * gm
        return (d * y).sum((-1, -2)) + (e.double() * x).sum((-1, -2))
    _, tol, _, tol_g = ref.backward64(dy, h, gamma, e)
    step = 1e-5   # the truncation error is of order step^2 and the rounding 1e-16 / step: both under 1e-9
    for i in range(4):
        eye = torch.zeros((96, 4, 96), dtype=torch.float64, device="cuda")
        eye[torch.arange(96), i, torch.arange(96)] = step
        num = (loss(x + eye, gm) - loss(x - eye, gm)) / (2 * step)
        ref.check(dh[i], num, tol[i] + 1e-9, "dh by differences")
    eye = torch.eye(96, dtype=torch.float64, device="cuda")[:, None] * step
    num = (loss(x, gm + eye) - loss(x, gm - eye)) / (2 * step)
    ref.check(dg, num, tol_g + 1e-8, "dgamma by differences")


def test_values_that_are_not_finite(ws):
    """A NaN row gives NaN gradients for that row alone (and for dgamma, which sums it)."""
    dy, h, gamma, e = inputs(2, 6, 128, 5)
    h[2, 5] = float("nan")
    dh, dg = run(ws, dy, h, gamma, e)
    assert dh[2].isnan().all() and dg.isnan().all()
    keep = [0, 1, 3, 4, 5]
    want, tol, _, _ = ref.backward64([t[keep] for t in dy], h[keep], gamma, e[keep])
    ref.check(dh[keep], want, tol, "dh")


def test_no_rows(ws):
    empty = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    dh, dg = run(ws, [empty], empty, torch.ones(256, device="cuda"), None)
    assert (dg == 0).all() and dh.shape == (0, 256)


def test_guards_and_stream(ws):
    """Rows behind the last and columns of other calls stay; a side stream."""
    dy, h, gamma, e = inputs(2, 5, 264, 8)
    buf = torch.full((8, 264), 3.0, dtype=torch.bfloat16, device="cuda")
    dgb = torch.full((300,), 9.0, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    are.allreduce_rmsnorm_backward(dy, h, gamma, ref.EPS, buf[:5], dgb[:264], ws, dres=e, stream=s)
    torch.cuda.synchronize()
    want, tol, want_g, tol_g = ref.backward64(dy, h, gamma, e)
    ref.check(buf[:5], want, tol, "dh")
    ref.check(dgb[:264], want_g, tol_g, "dgamma")
    assert (buf[5:] == 3).all() and (dgb[264:] == 9).all()


def test_graph_replays(ws):
    """Captured forward and backward of a step, replayed with new inputs."""
    R, M, N = 4, 320, 1024
    dy, h, gamma, e = inputs(R, M, N, 1)
    dh, dg = torch.empty_like(h), torch.empty(N, device="cuda")

    def call():
        are.allreduce_rmsnorm_backward(dy, h, gamma, ref.EPS, dh, dg, ws, dres=e)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(3):
        d2, h2, g2, e2 = inputs(R, M, N, 50 + k)
        for a, b in zip(dy + [h, gamma, e], d2 + [h2, g2, e2]):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        want, tol, want_g, tol_g = ref.backward64(dy, h, gamma, e)
        ref.check(dh, want, tol, "dh")
        ref.check(dg, want_g, tol_g, "dgamma")


def test_offsets_past_32_bits(ws):
    M, N = (1 << 18) + 5, 8200
    rows = [0, M // 2, M - 1]
    dy, h, gamma, _ = inputs(1, 3, N, 6, False)
    D = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    H = torch.ones((M, N), dtype=torch.bfloat16, device="cuda")
    D[rows], H[rows] = dy[0], h
    dh, dg = run(ws, [D], H, gamma, None)
    want, tol, want_g, tol_g = ref.backward64(dy, h, gamma, None)  # the other rows add exact zeros
    ref.check(dh[rows], want, tol, "dh")
    ref.check(dg, want_g, tol_g, "dgamma")
    assert (dh[1] == 0).all() and (dh[M - 2] == 0).all()


def test_refusals(ws):
    dy, h, gamma, e = inputs(2, 4, 256, 1)
    dh, dg = torch.empty_like(h), torch.empty(256, device="cuda")

    def call(dy=dy, h=h, gamma=gamma, dh=dh, dg=dg, w=ws, **k):
        are.allreduce_rmsnorm_backward(dy, h, gamma, k.pop("eps", ref.EPS), dh, dg, w, **k)
    for k in (dict(dy=[]), dict(dy=dy * 5), dict(h=h.float()), dict(h=h[:3]), dict(dh=dh[:, :128]), dict(dg=dg.double()),
              dict(dg=dg[:100]), dict(gamma=gamma.to(torch.bfloat16)), dict(dres=e.t()), dict(h=h.cpu())):
        with pytest.raises(ValueError):
            call(**k)
    for eps in (0.0, -1.0, float("inf")):
        with pytest.raises(are.AreError):
            call(eps=eps)
    wide = torch.zeros((1, 16392), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(are.AreError) as err:
        call([wide], wide, torch.ones(16392, device="cuda"), wide.clone(), None)
    assert err.value.status == are.EINVAL
    with are.Workspace(R_max=8, M_max=1, N_max=128) as small:
        with pytest.raises(are.AreError) as err:
            call(w=small)
        assert err.value.status == are.ECAPACITY


@pytest.mark.parametrize("N", [8, 64, 264, 768, 1032, 2048, 2056, 2816, 3592, 4096, 7680])
def test_workspaces_no_wider_than_the_row(N):
    """The partial sums of dgamma fit a workspace made for just this width, with as many blocks as a call can have."""
    need_gpu()
    dy, h, gamma, e = inputs(1, 3300, N, N, True)
    want, tol, want_g, tol_g = ref.backward64(dy, h, gamma, e)
    with are.Workspace(R_max=1, M_max=1, N_max=N) as small:
        dh, dg = run(small, dy, h, gamma, e)
        grid = small.last_launch()["grid"]
    ref.check(dh, want, tol, "dh")
    ref.check(dg, want_g, tol_g, "dgamma")
    assert grid >= 152 if N > 4096 else grid >= 304
