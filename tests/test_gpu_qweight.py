"""The few-token linear with 4-bit weights and group scales, summed over R ranks."""
import pytest
import torch

import all_reduce_epilogue_gb300 as are
from tests import ops_ref as ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    need_gpu()
    with are.Workspace(R_max=8, M_max=1, N_max=8) as w:
        yield w


def weights(R, N, K, group, zero, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    G = -(-K // group)
    out = []
    for _ in range(R):
        c = torch.randint(0, 256, (N, K // 2), generator=g, device="cuda", dtype=torch.uint8)
        s = (torch.rand((N, G), generator=g, device="cuda") * 0.02 + 0.001).to(torch.bfloat16)
        z = torch.randint(0, 16, (N, G), generator=g, device="cuda", dtype=torch.uint8) if zero else None
        out.append((c, s, z))
    return out, g


def tokens8(x, xgroup, pow2):
    xg = ref.grouped(x, xgroup)
    a = xg.abs().amax(-1)
    if pow2:
        s = ref.pow2_byte(a).to(torch.uint8)
        f = ref.e8m0_value(s)
    else:
        s = torch.where(a > 0, a / 448, 1.0).float()
        f = s.double()
    q = (xg / f[..., None]).flatten(-2)[..., :x.shape[-1]].float().clamp(-448, 448).to(torch.float8_e4m3fn)
    val = (ref.grouped(q.double(), xgroup) * f[..., None]).flatten(-2)[..., :x.shape[-1]]
    return q.contiguous(), s.contiguous(), val


def run(ws, x, w, group, xgroup=None, pow2=False, out=None):
    qw = [are.QWeight(*t, group) for t in w]
    M, N = x[0].shape[0], qw[0].N
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    if xgroup is None:
        are.gemm_ar_qweight(x, qw, out, ws)
        vals = x
    else:
        t = [tokens8(v.float(), xgroup, pow2) for v in x]
        are.gemm_ar_qweight_qx([v[0] for v in t], [v[1] for v in t], qw, out, ws, xgroup=xgroup)
        vals = [v[2] for v in t]
    assert ws.device_status()["code"] == 0
    return out, vals


# one token and one row of groups; ragged N, K and last groups; every token tile; K splits, several K tiles
SHAPES = [(1, 1, 8, 32), (2, 1, 256, 128), (8, 1, 1032, 2048), (1, 1, 4096, 4096), (3, 5, 136, 160), (4, 8, 520, 544),
          (5, 9, 264, 1056), (6, 16, 72, 800), (7, 17, 200, 288), (8, 33, 1000, 320), (8, 64, 136, 2080), (1, 64, 4104, 96),
          (2, 65, 128, 608), (1, 200, 72, 352), (1, 3, 16, 16384), (2, 20, 2048, 4128)]


@pytest.mark.parametrize("zero", [False, True])
@pytest.mark.parametrize("R,M,N,K", SHAPES)
def test_against_64_bits(ws, R, M, N, K, zero):
    for group in (32, 64, 128):
        w, g = weights(R, N, K, group, zero, R + M + N + K + group)
        x = [torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)]
        y, _ = run(ws, x, w, group)
        want, tol = ref.linear64(x, w, group)
        ref.check(y, want, tol, f"group {group}")
        assert ws.last_launch()["kernel"] == "qweight_kernel"


@pytest.mark.parametrize("xgroup,pow2", [(32, True), (64, False), (128, False), (128, True)])
@pytest.mark.parametrize("R,M,N,K", SHAPES)
def test_8_bit_tokens_against_64_bits(ws, R, M, N, K, xgroup, pow2):
    for group in (32, 128):
        w, g = weights(R, N, K, group, group == 32, R + M + N + K + group)
        x = [torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) * 3 for _ in range(R)]
        x[0][0] = 0
        y, vals = run(ws, x, w, group, xgroup, pow2)
        want, tol = ref.linear64(vals, w, group)
        ref.check(y, want, tol, f"group {group}")


def test_codes_enter_exactly(ws):
    """Integers in, integers out: one-hot tokens return columns of the weights, bit for bit."""
    N, K, group = 64, 256, 64
    w, _ = weights(1, N, K, group, True, 3)
    w[0][1].fill_(1.0)
    x = torch.zeros((64, K), dtype=torch.bfloat16, device="cuda")
    at = torch.randperm(K, device="cuda")[:64]
    x[torch.arange(64, device="cuda"), at] = 1
    y, _ = run(ws, [x], w, group)
    assert torch.equal(y.double(), ref.dequant64(*w[0], group)[:, at].T)


def test_outliers_and_extreme_scales(ws):
    """A token channel 10^4 times the others; group scales of 2^-100 and 2^20; a token of 10^30."""
    N, K, group = 40, 512, 128
    w, g = weights(2, N, K, group, True, 4)
    x = [torch.randn((5, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    x[0][:, 17] *= 1e4
    x[1][3] *= 1e30
    w[0][1][:, 1] = 2.0 ** -100
    w[1][1][5] = 2.0 ** 20
    y, _ = run(ws, x, w, group)
    want, tol = ref.linear64(x, w, group)
    ref.check(y, want, tol, "out")


def test_values_that_are_not_finite(ws):
    """A token's NaN or infinity stays in that token's outputs."""
    w, g = weights(2, 64, 256, 128, False, 5)
    w[0][0].fill_(0x99)  # every weight of rank 0: 1 * scale
    x = [torch.randn((6, 256), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    x[1][2, 100] = float("nan")
    x[0][4, 3] = float("inf")
    y, _ = run(ws, x, w, 128)
    assert y[2].isnan().all() and (y[4] == float("inf")).all()
    keep = [0, 1, 3, 5]
    want, tol = ref.linear64([t[keep] for t in x], w, 128)
    ref.check(y[keep], want, tol, "out")


def test_views_guards_stream_and_repeat(ws):
    R, M, N, K = 4, 3, 136, 320
    w, g = weights(R, N, K, 64, True, 6)
    x = [torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)]
    y, _ = run(ws, x, w, 64)
    big = [torch.full((M + 2, N), 5.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    are.gemm_ar_qweight(x, [are.QWeight(*t, 64) for t in w], [big[v % 2][:M] for v in range(R)], ws, stream=s)
    torch.cuda.synchronize()
    for b in big:
        assert torch.equal(b[:M], y) and (b[M:] == 5).all()


def test_graph_replays(ws):
    R, M, N, K = 8, 2, 1024, 512
    w, g = weights(R, N, K, 128, True, 7)
    qw = [are.QWeight(*t, 128) for t in w]
    x = [torch.zeros((M, K), dtype=torch.bfloat16, device="cuda") for _ in range(R)]
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    are.gemm_ar_qweight(x, qw, out, ws)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        are.gemm_ar_qweight(x, qw, out, ws)
    for _ in range(3):
        for t in x:
            t.normal_(generator=g)
        gr.replay()
        torch.cuda.synchronize()
        want, tol = ref.linear64(x, w, 128)
        ref.check(out, want, tol, "out")


def test_offsets_past_32_bits(ws):
    """More than 2^32 weights: the last rows."""
    N, K = (1 << 19) + 8, 8224
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    scale = torch.ones((N, 257), dtype=torch.bfloat16, device="cuda")
    w, g = weights(1, 16, K, 32, False, 8)
    codes[-16:], scale[-16:] = w[0][0], w[0][1]
    x = torch.randn((2, K), generator=g, device="cuda").to(torch.bfloat16)
    y, _ = run(ws, [x], [(codes, scale, None)], 32)
    want, tol = ref.linear64([x], w, 32)
    ref.check(y[:, -16:], want, tol, "last rows")


def test_empty(ws):
    w, _ = weights(2, 64, 128, 128, True, 9)
    x = [torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")] * 2
    assert run(ws, x, w, 128)[0].shape == (0, 64)
    z = are.QWeight(torch.empty((64, 0), dtype=torch.uint8, device="cuda"),
                    torch.empty((64, 0), dtype=torch.bfloat16, device="cuda"))
    out = torch.full((3, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    are.gemm_ar_qweight([torch.empty((3, 0), dtype=torch.bfloat16, device="cuda")], [z], out, ws)
    assert (out == 0).all() and ws.last_launch()["kernel"] == "memset"


def test_refusals(ws):
    w, g = weights(2, 64, 128, 128, True, 9)
    qw = [are.QWeight(*t, 128) for t in w]
    x = [torch.randn((3, 128), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2)]
    out = torch.empty((3, 64), dtype=torch.bfloat16, device="cuda")
    c, s, z = w[0]
    for a in ((c, s, z, 96), (c, s, z, 64), (c.int(), s, z, 128), (c, s.float(), z, 128), (c, s, z.int(), 128),
              (c, s, z[:3], 128), (c.t(), s, z, 128)):
        with pytest.raises(ValueError):
            are.QWeight(*a)
    for a in (([], qw, out), (x, qw[:1], out), (x[:1], qw, out), ([t.float() for t in x], qw, out),
              ([t[:, :96] for t in x], qw, out), (x, qw, out[:2]), (x, qw, out.float()), (x, qw, [out]),
              ([t.cpu() for t in x], qw, out)):
        with pytest.raises(ValueError):
            are.gemm_ar_qweight(*a, ws)
    odd = are.QWeight(torch.zeros((64, 24), dtype=torch.uint8, device="cuda"),
                      torch.ones((64, 1), dtype=torch.bfloat16, device="cuda"))
    with pytest.raises(are.AreError):  # K = 48
        are.gemm_ar_qweight([torch.zeros((3, 48), dtype=torch.bfloat16, device="cuda")], [odd], out, ws)
    xq = [t.to(torch.float8_e4m3fn) for t in x]
    xs = [torch.ones((3, 1), device="cuda") for _ in x]
    for a, k in (((xq, xs[:1], qw, out), {}), ((xq, xs, qw, out), dict(xgroup=64)), ((xq, xs, qw, out), dict(xgroup=16)),
                 ((x, xs, qw, out), {}), ((xq, [xs[0], xs[1].to(torch.uint8)], qw, out), {}),
                 ((xq, [t.double() for t in xs], qw, out), {})):
        with pytest.raises(ValueError):
            are.gemm_ar_qweight_qx(*a, ws, **k)


def test_zero_points_of_some_ranks(ws):
    """Ranks with and without zero points in one call (a CTA may take several ranks)."""
    for R, N, K in ((8, 72, 320), (8, 4096, 512), (3, 2048, 256)):
        w, g = weights(R, N, K, 64, True, R + N)
        w = [(c, s, z if r % 2 else None) for r, (c, s, z) in enumerate(w)]
        x = [torch.randn((2, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)]
        y, _ = run(ws, x, w, 64)
        want, tol = ref.linear64(x, w, 64)
        ref.check(y, want, tol, f"R {R}")


def test_tokens_of_any_magnitude(ws):
    """Tokens from bf16's smallest to near its largest values, each its own magnitude, and zeros."""
    w, g = weights(2, 64, 512, 128, True, 12)
    x = [torch.randn((9, 512), generator=g, device="cuda") for _ in range(2)]
    for i, e in enumerate((-130, -126, -100, -30, 0, 40, 100, 115)):
        for t in x:
            t[i] *= 2.0 ** e
    x[0][8], x[1][8] = 0, 0
    x = [t.to(torch.bfloat16) for t in x]
    y, _ = run(ws, x, w, 128)
    want, tol = ref.linear64(x, w, 128)
    ref.check(y, want, tol + 2.0 ** -133, "out")  # bf16's smallest step


@pytest.mark.parametrize("M", [1, 9, 40])
def test_power_of_two_scales_of_any_size(ws, M):
    """E8M0 token scales that differ by 2^40 within a row, the smallest and large ones, NaN scales and NaN codes."""
    R, N, K, group = 2, 72, 544, 128
    w, g = weights(R, N, K, group, True, 21 + M)
    qw = [are.QWeight(*t, group) for t in w]
    xq = [torch.randint(0, 256, (M, K), generator=g, device="cuda", dtype=torch.uint8) for _ in range(R)]
    for q in xq:
        q[(q & 0x7F) == 0x7F] = 0x38
    xs = [torch.randint(107, 148, (M, 17), generator=g, device="cuda", dtype=torch.uint8) for _ in range(R)]
    xs[0][0, :9] = 3            # 2^-124
    xs[1][0, :] = 5
    xs[0][M // 2, 11] = 230     # 2^103
    nan = []
    if M > 1:
        xs[1][M - 1, 16] = 255  # the last, short group's scale is NaN
        xq[0][1, 100] = 0xFF    # a NaN code
        nan = [1, M - 1]
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    are.gemm_ar_qweight_qx(xq, xs, qw, out, ws, xgroup=32)
    val = [q.view(torch.float8_e4m3fn).double() * ref.e8m0_value(f).repeat_interleave(32, -1)[:, :K] for q, f in zip(xq, xs)]
    want, tol = ref.linear64(val, w, group)
    keep = [i for i in range(M) if i not in nan]
    assert out[nan].isnan().all()
    ref.check(out[keep], want[keep], tol[keep] + 2.0 ** -133, "out")


@pytest.mark.parametrize("M", [12, 40])
def test_values_that_are_not_finite_in_wide_tiles(ws, M):
    """NaN and infinities in the first, a middle and the last token and k of staged tiles."""
    R, N, K = 3, 72, 832
    w, g = weights(R, N, K, 64, False, 31 + M)
    w[0][0].fill_(0x99)  # every weight of rank 0: 1 * scale
    x = [torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)]
    x[0][0, 0] = float("-inf")
    x[2][M // 2, 255] = float("nan")
    x[0][M - 1, K - 1] = float("inf")
    x[0][M - 1, 256] = float("inf")
    y, _ = run(ws, x, w, 64)
    assert (y[0] == float("-inf")).all() and y[M // 2].isnan().all() and (y[M - 1] == float("inf")).all()
    keep = [m for m in range(M) if m not in (0, M // 2, M - 1)]
    want, tol = ref.linear64([t[keep] for t in x], w, 64)
    ref.check(y[keep], want, tol, "out")


@pytest.mark.parametrize("M,N,K", [(300, 72, 4096), (20, 64, 32768), (9, 40, 40000), (70, 24, 20000)])
@pytest.mark.parametrize("eight", [False, True])
def test_more_tokens_than_the_staging_buffer_holds(M, N, K, eight):
    """A workspace for one rank: tokens that go in several parts, and rows too long to be staged at all."""
    need_gpu()
    with are.Workspace(R_max=1, M_max=1, N_max=8) as small:
        w, g = weights(1, N, K, 32, True, M + K)
        x = [torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)]
        big = torch.full((M + 1, N), 5.0, dtype=torch.bfloat16, device="cuda")
        _, vals = run(small, x, w, 32, 32 if eight else None, False, out=big[:M])
        want, tol = ref.linear64(vals, w, 32)
        ref.check(big[:M], want, tol, "out")
        assert (big[M] == 5).all()


def test_operands_written_just_before(ws):
    """Weights, scales and tokens that the kernel before in the stream writes, call after call into the same buffers."""
    for M in (2, 16, 40):
        R, N, K = 4, 512, 1024
        sets = [weights(R, N, K, 128, True, 50 + i)[0] for i in range(3)]
        g = torch.Generator(device="cuda").manual_seed(M)
        xs = [[torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)] for _ in range(3)]
        w = [tuple(torch.zeros_like(t) for t in r) for r in sets[0]]
        qw = [are.QWeight(*t, 128) for t in w]
        x = [torch.zeros_like(t) for t in xs[0]]
        outs = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(9)]

        def step(i, out):
            for r in range(R):
                for to, of in zip(w[r], sets[i % 3][r]):
                    to.copy_(of)
                x[r].copy_(xs[i * 2 % 3][r])
            are.gemm_ar_qweight(x, qw, out, ws)

        for i in range(3):  # with time in between
            step(i, outs[i])
            torch.cuda.synchronize()
        want = [o.clone() for o in outs[:3]]
        for i in range(9):
            step(i, outs[i])
        torch.cuda.synchronize()
        assert all(torch.equal(outs[i], want[i % 3]) for i in range(9))
        for o in outs:
            o.zero_()
        gr = torch.cuda.CUDAGraph()
        with torch.cuda.graph(gr):
            for i in range(9):
                step(i, outs[i])
        for _ in range(2):
            gr.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(outs[i], want[i % 3]) for i in range(9))


def test_calls_in_a_row_share_the_staging_buffer(ws):
    """Different layers back to back, by themselves and as two captured graphs: each sees its own tokens."""
    layers = []
    for i, (R, M, N, K, group) in enumerate([(8, 16, 256, 512, 64), (2, 40, 520, 1056, 32), (8, 33, 72, 2048, 128),
                                             (1, 10, 1024, 256, 128), (3, 5, 136, 160, 32)]):
        w, g = weights(R, N, K, group, True, 70 + i)
        x = [torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)]
        out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
        layers.append(([are.QWeight(*t, group) for t in w], x, out, ref.linear64(x, w, group)))

    def step(ls):
        for qw, x, out, _ in ls:
            are.gemm_ar_qweight(x, qw, out, ws)

    def look():
        torch.cuda.synchronize()
        for _, _, out, (want, tol) in layers:
            ref.check(out, want, tol, "out")
            out.zero_()

    for _ in range(3):
        step(layers)
    look()
    graphs = []
    for part in (layers[:3], layers[3:]):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            step(part)
    for _ in range(3):
        for gr in graphs:
            gr.replay()
    look()


def test_refuses_ranks_without_weights(ws):
    w, _ = weights(2, 16, 64, 32, False, 90)
    x = [torch.zeros((2, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    out = torch.full((2, 16), 3.0, dtype=torch.bfloat16, device="cuda")
    for qw in ([], [are.QWeight(*w[0], 32)], [are.QWeight(*t, 32) for t in w + w[:1]]):
        with pytest.raises(ValueError):
            are.gemm_ar_qweight(x, qw, out, ws)
    torch.cuda.synchronize()
    assert (out == 3).all()


@pytest.fixture(params=[8, 16, 32], ids=lambda t: f"tiles of {t}")
def tiled(request):
    """A workspace whose calls all take tiles of so many tokens."""
    need_gpu()
    with are.Workspace(R_max=8, M_max=1, N_max=8) as w:
        w.set_debug(are.DEBUG_QWEIGHT_FEW if request.param == 8 else are.DEBUG_QWEIGHT_STAGED, request.param)
        yield w, {8: 1, 16: 2, 32: 4}[request.param]


TILED = [(1, 1, 8, 32), (2, 3, 256, 128), (5, 9, 264, 1056), (6, 16, 72, 800), (7, 17, 200, 288), (8, 33, 1000, 320),
         (8, 64, 136, 2080), (1, 64, 4104, 96), (2, 65, 128, 608), (1, 100, 72, 352), (2, 20, 2048, 4128), (4, 31, 32, 64)]


@pytest.mark.parametrize("R,M,N,K", TILED)
def test_every_tile_against_64_bits(tiled, R, M, N, K):
    w_, variant = tiled
    for group in (32, 64, 128):
        w, g = weights(R, N, K, group, group != 64, R + M + N + K + group)
        x = [torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)]
        for xgroup, pow2 in ((None, False), (32, True), (32, False), (64, False), (128, True), (128, False)):
            y, vals = run(w_, x, w, group, xgroup, pow2)
            want, tol = ref.linear64(vals, w, group)
            ref.check(y, want, tol, f"group {group}, token group {xgroup}, {pow2}")
        assert w_.last_launch()["variant"] == variant


def test_every_tile_with_values_that_are_not_finite(tiled):
    w_, _ = tiled
    R, M, N, K = 3, 40, 72, 832
    w, g = weights(R, N, K, 64, False, 71)
    w[0][0].fill_(0x99)  # every weight of rank 0: 1 * scale
    x = [torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)]
    x[0][0, 0] = float("-inf")
    x[2][M // 2, 255] = float("nan")
    x[0][M - 1, K - 1] = float("inf")
    y, _ = run(w_, x, w, 64)
    assert (y[0] == float("-inf")).all() and y[M // 2].isnan().all() and (y[M - 1] == float("inf")).all()
    keep = [m for m in range(M) if m not in (0, M // 2, M - 1)]
    want, tol = ref.linear64([t[keep] for t in x], w, 64)
    ref.check(y[keep], want, tol, "out")


def test_every_tile_captured_with_operands_written_before(tiled):
    w_, _ = tiled
    R, M, N, K = 4, 40, 512, 1024
    sets = [weights(R, N, K, 128, True, 80 + i) for i in range(2)]
    xs = [[torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)] for _, g in sets]
    w = [tuple(torch.zeros_like(t) for t in r) for r in sets[0][0]]
    qw, x = [are.QWeight(*t, 128) for t in w], [torch.zeros_like(t) for t in xs[0]]
    outs = [torch.empty((M, N), dtype=torch.bfloat16, device="cuda") for _ in range(4)]

    def step(i):
        for r in range(R):
            for to, of in zip(w[r], sets[i % 2][0][r]):
                to.copy_(of)
            x[r].copy_(xs[i % 2][r])
        are.gemm_ar_qweight(x, qw, outs[i], w_)

    for i in range(4):
        step(i)
    gr = torch.cuda.CUDAGraph()
    with torch.cuda.graph(gr):
        for i in range(4):
            step(i)
    for _ in range(2):
        for i in range(4):
            want, tol = ref.linear64(xs[i % 2], sets[i % 2][0], 128)
            ref.check(outs[i], want, tol, f"call {i}")
        for o in outs:
            o.zero_()
        gr.replay()
