"""All-reduce + residual + LayerNorm and its backward pass."""
import pytest
import torch

import all_reduce_epilogue_gb300 as are
from tests import ends_ref as ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    need_gpu()
    with are.Workspace(R_max=8, M_max=1, N_max=16384) as w:
        yield w


def randn(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, device="cuda")


def inputs(R, M, N, seed, residual=True, shift=0.0):
    r = randn(seed)
    parts = [(r(M, N) + shift).to(torch.bfloat16) for _ in range(R)]
    res = (r(M, N) + 3 * r(M, 1)).to(torch.bfloat16) if residual else None
    return parts, res, 1 + 0.1 * r(N), 0.1 * r(N)


def run(ws, parts, res, gamma, beta, residual_out=True, out=None):
    M, N = parts[0].shape
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    ro = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda") if residual_out else None
    are.allreduce_layernorm(parts, res, gamma, beta, ref.EPS, out, ws, residual_out=ro)
    assert ws.device_status()["code"] == 0
    return out, ro


# one token to several rows a block; one pack, a partial last warp, every packs-per-thread variant, the widest row
SHAPES = [(1, 1, 8), (2, 3, 40), (8, 1, 7168), (3, 5, 264), (4, 37, 4104), (8, 310, 1024), (1, 700, 2056), (5, 2, 5000),
          (8, 2, 8192), (2, 3, 10008), (7, 2, 16384), (8, 2, 32768), (1, 1300, 64), (6, 200, 7168), (2, 160, 4096),
          (1, 152, 2064), (4, 153, 5000), (3, 400, 8192), (8, 320, 16384), (1, 400, 24000), (8, 170, 32768), (1, 4000, 768),
          # lanes a row: 1 to 16 packs with any number of ranks, up to 128 with few, a last warp with rows missing
          (1, 700, 8), (8, 1111, 64), (3, 611, 72), (5, 701, 128), (1, 5001, 136), (2, 5003, 264), (1, 5000, 520), (2, 4871, 768),
          (1, 6001, 1000), (1, 5000, 1024)]


@pytest.mark.parametrize("R,M,N", SHAPES)
def test_forward_against_64_bits(ws, R, M, N):
    parts, res, gamma, beta = inputs(R, M, N, 1000 * R + M + N)
    if M > 4:
        for t in parts:
            t[2] = 0
        res[2] = 0       # a padded row: xhat = 0, y = beta
    y, ro = run(ws, parts, res, gamma, beta)
    want, tol, h, tol_h = ref.layernorm64(parts, res, gamma, beta)
    ref.check(y, want, tol, "y")
    ref.check(ro, h, tol_h, "residual_out")
    assert ws.last_launch()["kernel"] in ("layernorm_rows_kernel", "layernorm_narrow_kernel")
    # without the optional tensors; in place of the residual
    y2, _ = run(ws, parts, res, gamma, beta, residual_out=False)
    assert torch.equal(y2, y)
    into, out = res.clone(), torch.empty_like(y)
    are.allreduce_layernorm(parts, into, gamma, beta, ref.EPS, out, ws, residual_out=into)
    assert torch.equal(into, ro) and torch.equal(out, y)
    y3, ro3 = run(ws, parts, None, gamma, None)
    want, tol, h, tol_h = ref.layernorm64(parts, None, gamma, None)
    ref.check(y3, want, tol, "y, no residual, no beta")
    ref.check(ro3, h, tol_h, "residual_out, no residual")


@pytest.mark.parametrize("N", [64, 1000, 7168])
def test_mean_large_against_the_spread(ws, N):
    """Rows of 1000 +- 4: the squares' mean less the mean's square would lose 1.6e-5 of 1e6."""
    parts, _, gamma, beta = inputs(1, 20, N, N, shift=0)
    parts[0] = (parts[0].float() * 4 + 1000).to(torch.bfloat16)
    y, _ = run(ws, parts, None, gamma, beta)
    want, tol, _, _ = ref.layernorm64(parts, None, gamma, beta)
    assert (tol < 0.05 * (1 + want.abs())).all()   # the bound says something
    ref.check(y, want, tol, "y")
    constant = [torch.full((3, N), 1000.0, dtype=torch.bfloat16, device="cuda")]
    y, _ = run(ws, constant, None, gamma, beta)
    # xhat is the mean's rounding error, 1000 * 64 U at most, over sqrt(eps)
    bound = 1000 * 64 * ref.U / ref.EPS ** 0.5 * gamma.abs() + ref.BF16 * (beta.abs() + 2) + 1e-3
    assert ((y.double() - beta.double()).abs() <= bound).all()


def test_values_that_are_not_finite(ws):
    parts, res, gamma, beta = inputs(2, 6, 136, 5)
    parts[0][1, 7] = float("nan")
    parts[1][4, 100] = float("inf")
    y, ro = run(ws, parts, res, gamma, beta)
    assert y[1].isnan().all() and y[4].isnan().all() and ro[1, 7].isnan() and ro[4, 100].isinf()
    keep = [0, 2, 3, 5]
    want, tol, _, _ = ref.layernorm64([t[keep] for t in parts], res[keep], gamma, beta)
    ref.check(y[keep], want, tol, "y")


def test_negative_zero_and_guards(ws):
    """A sum of -0.0 counts as +0.0 (residual_out's bits); rows behind the last stay; a side stream."""
    x = torch.full((5, 264), -0.0, dtype=torch.bfloat16, device="cuda")
    gamma, beta = torch.ones(264, device="cuda"), torch.zeros(264, device="cuda")
    buf, ro = (torch.full((8, 264), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    are.allreduce_layernorm([x, x], None, gamma, beta, ref.EPS, buf[:5], ws, residual_out=ro[:5], stream=s)
    torch.cuda.synchronize()
    assert (buf[:5] == 0).all() and (ro[:5].view(torch.int16) == 0).all()
    assert (buf[5:] == 3).all() and (ro[5:] == 3).all()


def backward_inputs(R, M, N, seed, dres=True):
    r = randn(seed)
    dy = [(r(M, N) * 0.01).to(torch.bfloat16) for _ in range(R)]
    return (dy, (r(M, N) * 3 + 2 * r(M, 1)).to(torch.bfloat16), 1 + 0.1 * r(N),
            (r(M, N) * 0.01).to(torch.bfloat16) if dres else None)


def backward(ws, dy, h, gamma, dres, dgamma=True, dbeta=True, dh=None):
    M, N = h.shape
    dh = torch.empty((M, N), dtype=torch.bfloat16, device="cuda") if dh is None else dh
    dg = torch.full((N,), 7.0, device="cuda") if dgamma else None
    db = torch.full((N,), 7.0, device="cuda") if dbeta else None
    are.allreduce_layernorm_backward(dy, h, gamma, ref.EPS, dh, dg, db, ws, dres=dres)
    assert ws.device_status()["code"] == 0
    return dh, dg, db


@pytest.mark.parametrize("R,M,N,dres", [(1, 1, 8, True), (8, 1, 7168, True), (2, 2, 40, False), (3, 7, 264, True),
                                        (1, 151, 1024, True), (1, 1000, 2048, False), (5, 305, 2056, True),
                                        (4, 33, 4096, False), (8, 620, 4104, True), (3, 9, 5000, True), (8, 311, 7168, True),
                                        (8, 2, 8192, False), (2, 160, 8200, True), (8, 157, 16384, True), (1, 2500, 64, True),
                                        (1, 400, 7680, True), (3, 200, 7688, False), (4, 170, 11528, True), (1, 160, 15368, True),
                                        (1, 320, 16384, True), (1, 310, 11520, True),
                                        # lanes a row: 1 to 16 packs with any number of ranks, up to 64 with one, a last warp
                                        # with rows missing
                                        (1, 1300, 8, True), (8, 1303, 64, True), (3, 1221, 72, False), (5, 2001, 128, True),
                                        (1, 1301, 136, True), (1, 5003, 264, False), (1, 3001, 512, True), (2, 1301, 264, True)])
def test_backward_against_64_bits(ws, R, M, N, dres):
    dy, h, gamma, e = backward_inputs(R, M, N, 100 * R + M + N, dres)
    if M > 4:
        h[3] = 0              # a padded row: inv = eps^-1/2
        for t in dy:
            t[2] = 0
    got = backward(ws, dy, h, gamma, e)
    want = ref.layernorm_backward64(dy, h, gamma, e)
    for g, w, tol, what in zip(got, want[::2], want[1::2], ("dh", "dgamma", "dbeta")):
        ref.check(g, w, tol, what)
    assert ws.last_launch()["kernel"] in ("layernorm_backward_rows_kernel", "layernorm_backward_narrow_kernel")
    for a, b in zip(got, backward(ws, dy, h, gamma, e)):
        assert torch.equal(a, b)
    # frozen weights and an in-place residual gradient give the same bits
    into = e.clone() if dres else None
    dh2, none, db2 = backward(ws, dy, h, gamma, into, dgamma=False, dh=into)
    assert none is None and torch.equal(dh2, got[0]) and torch.equal(db2, got[2])
    dh3, dg3, _ = backward(ws, dy, h, gamma, e, dbeta=False)
    assert torch.equal(dh3, got[0]) and torch.equal(dg3, got[1])
    assert torch.equal(backward(ws, dy, h, gamma, e, False, False)[0], got[0])


@pytest.mark.parametrize("R", [1, 3])
@pytest.mark.parametrize("N", [64, 264, 1000, 2056, 4096, 7168, 16384])
def test_backward_of_means_large_against_the_spread(ws, N, R):
    """Rows of 1000 +- 4 between rows of 3 +- 3 (next to the border of the two formulas) and 0 +- 3: the first kind is summed
    again around its mean, and neither kind changes its bits with what its neighbours are."""
    M = 1500
    dy, h, gamma, e = backward_inputs(R, M, N, 3 * N + R)
    x = h.float() / 3
    kind = torch.arange(M, device="cuda") % 3
    near = torch.where(kind[:, None] == 0, x * 3 + 6, x * 3).to(torch.bfloat16)
    h = torch.where(kind[:, None] == 2, (x * 4 + 1000).to(torch.bfloat16), near)
    got = backward(ws, dy, h, gamma, e)
    want = ref.layernorm_backward64(dy, h, gamma, e)
    for g, w, tol, what in zip(got, want[::2], want[1::2], ("dh", "dgamma", "dbeta")):
        ref.check(g, w, tol, what)
    alone = backward(ws, dy, near, gamma, e)[0]
    assert torch.equal(alone[kind != 2], got[0][kind != 2])


def test_backward_against_differences(ws):
    """The gradient of L = sum(dy * y) + sum(dres * h) by central differences of the forward formula in 64 bits."""
    dy, h, gamma, e = backward_inputs(3, 4, 96, 77)
    dh, dg, db = backward(ws, dy, h, gamma, e)
    d, x, gm = sum(t.double() for t in dy), h.double(), gamma.double()

    def loss(x, gm, bt):
        c = x - x.mean(-1, keepdim=True)
        y = c / torch.sqrt((c * c).mean(-1, keepdim=True) + ref.EPS) * gm + bt
        return (d * y).sum((-1, -2)) + (e.double() * x).sum((-1, -2))
    _, tol, _, tol_g, _, tol_b = ref.layernorm_backward64(dy, h, gamma, e)
    step = 1e-5   # the truncation error is of order step^2 and the rounding 1e-16 / step: both under 1e-9
    for i in range(4):
        eye = torch.zeros((96, 4, 96), dtype=torch.float64, device="cuda")
        eye[torch.arange(96), i, torch.arange(96)] = step
        ref.check(dh[i], (loss(x + eye, gm, 0) - loss(x - eye, gm, 0)) / (2 * step), tol[i] + 1e-9, "dh by differences")
    eye = torch.eye(96, dtype=torch.float64, device="cuda")[:, None] * step
    ref.check(dg, (loss(x, gm + eye, 0) - loss(x, gm - eye, 0)) / (2 * step), tol_g + 1e-8, "dgamma by differences")
    ref.check(db, (loss(x, gm, eye) - loss(x, gm, -eye)) / (2 * step), tol_b + 1e-8, "dbeta by differences")


def test_backward_of_a_nan_row_and_of_no_rows(ws):
    dy, h, gamma, e = backward_inputs(2, 6, 128, 5)
    h[2, 5] = float("nan")
    dh, dg, db = backward(ws, dy, h, gamma, e)
    assert dh[2].isnan().all() and dg.isnan().all()
    keep = [0, 1, 3, 4, 5]
    want = ref.layernorm_backward64([t[keep] for t in dy], h[keep], gamma, e[keep])
    ref.check(dh[keep], want[0], want[1], "dh")
    want = ref.layernorm_backward64(dy, torch.zeros_like(h), gamma, e)
    ref.check(db, want[4], want[5], "dbeta")
    empty = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    dh, dg, db = backward(ws, [empty], empty, torch.ones(256, device="cuda"), None)
    assert (dg == 0).all() and (db == 0).all()
    run(ws, [empty], None, torch.ones(256, device="cuda"), None)


def test_graph_replays_of_both(ws):
    """Captured forward and backward, replayed with new inputs."""
    R, M, N = 4, 320, 1024
    parts, res, gamma, beta = inputs(R, M, N, 1)
    dy, _, _, e = backward_inputs(R, M, N, 2)
    y, h, dh = (torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(3))
    dg, db = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")

    def call():
        are.allreduce_layernorm(parts, res, gamma, beta, ref.EPS, y, ws, residual_out=h)
        are.allreduce_layernorm_backward(dy, h, gamma, ref.EPS, dh, dg, db, ws, dres=e)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(3):
        for a, b in zip(parts + [res, gamma, beta], [*inputs(R, M, N, 50 + k)[0], *inputs(R, M, N, 50 + k)[1:]]):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        want, tol, _, _ = ref.layernorm64(parts, res, gamma, beta)
        ref.check(y, want, tol, "y")
        want = ref.layernorm_backward64(dy, h, gamma, e)
        for got, w, tol in zip((dh, dg, db), want[::2], want[1::2]):
            ref.check(got, w, tol, "gradient")


@pytest.mark.parametrize("N", [8, 64, 264, 2048, 2056, 4096, 16384])
def test_workspaces_no_wider_than_the_row(N):
    """Partial sums of every block fit a workspace made for this width."""
    need_gpu()
    dy, h, gamma, e = backward_inputs(1, 3100, N, N)
    with are.Workspace(R_max=1, M_max=1, N_max=N) as w:
        got = backward(w, dy, h, gamma, e)
    want = ref.layernorm_backward64(dy, h, gamma, e)
    for g, v, tol in zip(got, want[::2], want[1::2]):
        ref.check(g, v, tol, "gradient")


def test_offsets_past_32_bits(ws):
    M, N = (1 << 18) + 5, 8200
    rows = [0, M // 2, M - 1]
    r = randn(3)
    x = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    x[rows] = r(3, N).to(torch.bfloat16)
    gamma, beta = 1 + 0.1 * r(N), 0.1 * r(N)
    out = torch.empty_like(x)
    are.allreduce_layernorm([x], None, gamma, beta, ref.EPS, out, ws)
    want, tol, _, _ = ref.layernorm64([x[rows]], None, gamma, beta)
    ref.check(out[rows], want, tol, "y")
    assert (out[1] == beta.to(torch.bfloat16)).all()
    dg, db = torch.empty(N, device="cuda"), torch.empty(N, device="cuda")
    dy = [x]
    are.allreduce_layernorm_backward(dy, x, gamma, ref.EPS, out, dg, db, ws)
    want = ref.layernorm_backward64([x[rows]], x[rows], gamma, None)
    for g, v, tol in zip((out[rows], dg, db), want[::2], want[1::2]):
        ref.check(g, v, tol + 1e-12, "gradient")
    assert ws.device_status()["code"] == 0


def test_refusals(ws):
    parts, res, gamma, beta = inputs(2, 3, 64, 1)
    out, dg = torch.empty_like(res), torch.empty(64, device="cuda")
    bad = [dict(partials=[]), dict(partials=[parts[0], parts[1][:2]]), dict(gamma=gamma.to(torch.bfloat16)), dict(beta=beta[:32]),
           dict(out=out.float()), dict(residual=res.t()), dict(residual_out=out[:, :32]), dict(partials=[parts[0].cpu()])]
    for b in bad:
        kw = dict(partials=parts, residual=res, gamma=gamma, beta=beta, out=out, residual_out=None)
        kw.update(b)
        with pytest.raises(ValueError):
            are.allreduce_layernorm(kw["partials"], kw["residual"], kw["gamma"], kw["beta"], ref.EPS, kw["out"], ws,
                                    residual_out=kw["residual_out"])
    for eps in (0.0, -1.0, float("nan"), float("inf")):
        with pytest.raises(are.AreError):
            are.allreduce_layernorm(parts, res, gamma, beta, eps, out, ws)
        with pytest.raises(are.AreError):
            are.allreduce_layernorm_backward(parts, res, gamma, eps, out, dg, dg.clone(), ws)
    odd = torch.empty((3, 60), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(are.AreError):
        are.allreduce_layernorm([odd], None, torch.ones(60, device="cuda"), None, ref.EPS, odd, ws)
    with pytest.raises(ValueError):
        are.allreduce_layernorm_backward(parts, res, gamma, ref.EPS, out, dg, dg[:8], ws)
    with are.Workspace(R_max=1, M_max=1, N_max=32) as small:
        with pytest.raises(are.AreError):
            are.allreduce_layernorm(parts, res, gamma, beta, ref.EPS, out, small)   # R
        with pytest.raises(are.AreError):
            are.allreduce_layernorm_backward(parts[:1], res, gamma, ref.EPS, out, dg, None, small)  # N


@pytest.mark.parametrize("R,M,N", [(2, 700, 64), (1, 5001, 264), (3, 37, 4104), (1, 153, 24000)])
def test_in_place_of_an_input(ws, R, M, N):
    """`out` may be a partial or the residual itself: a row is read before it is written."""
    parts, res, gamma, beta = inputs(R, M, N, R + M + N)
    y, ro = run(ws, parts, res, gamma, beta)
    into = res.clone()
    run(ws, parts, into, gamma, beta, out=into)
    assert torch.equal(into, y)
    first = parts[0].clone()
    _, h = run(ws, [first] + parts[1:], res, gamma, beta, out=first)
    assert torch.equal(first, y) and torch.equal(h, ro)


def test_overlaps_are_refused(ws):
    """Memory that a call writes next to what it reads: every other overlap than an input in place."""
    M, N = 6, 64
    buf = torch.zeros(4 * M * N, dtype=torch.bfloat16, device="cuda")
    at = lambda k: buf[k:k + M * N].view(M, N)
    x, shifted, free = at(0), at(8), at(2 * M * N)
    sums = torch.zeros(3 * N, device="cuda")
    gamma, a, b = sums[:N], sums[N:2 * N], sums[2 * N:]

    def forward(parts, res, out, ro, beta=a, weight=gamma):
        are.allreduce_layernorm(parts, res, weight, beta, ref.EPS, out, ws, residual_out=ro)

    def back(dy, h, dh, dgamma=a, dbeta=b, dres=None):
        are.allreduce_layernorm_backward(dy, h, gamma, ref.EPS, dh, dgamma, dbeta, ws, dres=dres)

    other = torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")
    words = buf.view(torch.float32)[:N]   # in x
    for call in (lambda: forward([x], None, shifted, None), lambda: forward([x], shifted, other, x),
                 lambda: forward([x], other, free, shifted), lambda: forward([x], None, free, free),
                 lambda: forward([other], x, other, shifted), lambda: forward([other], None, x, None, beta=words),
                 lambda: forward([other], None, other, x, weight=words),
                 lambda: back([x], other, x), lambda: back([x], other, shifted), lambda: back([other], x, x),
                 lambda: back([other], x, free, dres=at(2 * M * N + 8)), lambda: back([x], other, free, dgamma=a, dbeta=a),
                 lambda: back([x], other, free, dgamma=gamma), lambda: back([x], other, free, dbeta=words)):
        with pytest.raises(are.AreError):
            call()
    back([x], other, free, dres=free)
    torch.cuda.synchronize()


@pytest.mark.parametrize("R,M,N,dres", [(3, 3100, 4104, True), (1, 5100, 5376, False), (8, 1700, 4608, True), (1, 155, 8192, True),
                                        (1, 500, 7688, False), (2, 155, 8192, True), (1, 153, 8200, True)])
def test_backward_of_wide_rows_against_64_bits(ws, R, M, N, dres):
    """Three packs a thread and two blocks an SM, where there are many rows; two packs and 16 warps with one rank."""
    test_backward_against_64_bits(ws, R, M, N, dres)


@pytest.mark.parametrize("R,M,N", [(2, 400, 8200), (1, 310, 12288), (8, 155, 10000), (1, 2500, 5000), (3, 600, 5000), (1, 600, 1032),
                                   (3, 310, 2048), (2, 160, 12296), (1, 309, 8192), (4, 311, 6144)])
def test_forward_of_every_split_of_a_row(ws, R, M, N):
    """Two to four packs a thread, one to four blocks an SM."""
    test_forward_against_64_bits(ws, R, M, N)
