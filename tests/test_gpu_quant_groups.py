"""AR + residual + RMSNorm with FP8 codes and a scale per group of columns."""
import pytest
import torch

import all_reduce_epilogue_gb300 as are
from tests import ops_ref as ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


def inputs(R, M, N, seed, residual=True):
    g = torch.Generator(device="cuda").manual_seed(seed)
    parts = [torch.randn((M, N), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)]
    res = torch.randn((M, N), generator=g, device="cuda").to(torch.bfloat16) if residual else None
    gamma = 1 + 0.1 * torch.randn(N, generator=g, device="cuda")
    return parts, res, gamma


def outputs(M, N, group, pow2):
    q = torch.full((M, N), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((M, -(-N // group)), 77, dtype=torch.uint8 if pow2 else torch.float32, device="cuda")
    return q, s


@pytest.fixture(scope="module")
def ws():
    need_gpu()
    with are.Workspace(R_max=8, M_max=64, N_max=8192) as w:
        yield w


def run(ws, parts, res, gamma, group, pow2, residual_out=True):
    M, N = parts[0].shape
    q, s = outputs(M, N, group, pow2)
    ro = torch.empty((M, N), dtype=torch.bfloat16, device="cuda") if residual_out else None
    are.allreduce_rmsnorm_quant_groups(parts, res, gamma, ref.EPS, q, s, ws, group=group, residual_out=ro)
    assert ws.device_status()["code"] == 0
    return q, s, ro


# one token to several rows a block; one pack, a partial last group, every packs-per-thread variant, widest row
SHAPES = [(1, 1, 8), (2, 3, 40), (8, 1, 7168), (3, 5, 264), (4, 37, 4104), (8, 310, 1024), (1, 700, 2056), (5, 2, 5000),
          (8, 2, 8192), (2, 3, 10008), (7, 2, 16384), (8, 2, 32768), (1, 1300, 64), (6, 200, 7168), (2, 160, 4096),
          (1, 152, 2064), (4, 153, 5000), (3, 400, 8192), (8, 320, 16384)]


@pytest.mark.parametrize("pow2", [False, True])
@pytest.mark.parametrize("R,M,N", SHAPES)
def test_against_64_bits(ws, R, M, N, pow2):
    for group in (32, 64, 128):
        parts, res, gamma = inputs(R, M, N, 1000 * R + M + N + group, residual=group != 64)
        q, s, ro = run(ws, parts, res, gamma, group, pow2)
        h, _, y, tol = ref.norm64(parts, res, gamma)
        ref.check_quant(q, s, y, tol, group, pow2)
        mag = sum(p.double().abs() for p in parts) + (res.double().abs() if res is not None else 0)
        ref.check(ro, h, ref.BF16 * h.abs() + (R + 1) * ref.U * mag * 1.01, "residual_out")
        assert ws.last_launch()["kernel"] == "norm_quant_rows_kernel"


@pytest.mark.parametrize("R,M,N,residual", [(8, 3, 7168, True), (3, 200, 1024, False), (1, 4, 4096, True)])
def test_residual_out_bits_equal_the_row_scaled_form(R, M, N, residual):
    need_gpu()
    parts, res, gamma = inputs(R, M, N, 5, residual)
    for t in parts:
        t[0, :64] = -0.0
    if residual:
        res[0, :32] = -0.0
    out, a = torch.empty_like(parts[0]), torch.empty_like(parts[0])
    with are.Workspace(R_max=8, M_max=M, N_max=N) as w:
        are.allreduce_add_rmsnorm(parts, res, gamma, ref.EPS, out, a, w)
        b = run(w, parts, res, gamma, 128, False)[2]
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))


@pytest.mark.parametrize("pow2", [False, True])
def test_zero_rows_and_tiny_values(ws, pow2):
    """Groups of zeros have scale 1; gamma takes y below the smallest normal scale."""
    parts, res, gamma = inputs(2, 4, 512, 9)
    for t in parts + [res]:
        t[1] = 0
    gamma[128:256] = 1e-39   # y ~ 1e-39, a denormal
    gamma[256:384] = 0
    gamma[384:] = 3e35
    q, s, ro = run(ws, parts, res, gamma, 128, pow2)
    assert (q[1] & 0x7F == 0).all() and (s[1] == (127 if pow2 else 1)).all()
    assert (s[:, 2] == (127 if pow2 else 1)).all() and (q[:, 256:384] & 0x7F == 0).all()
    h, _, y, tol = ref.norm64(parts, res, gamma)
    ref.check_quant(q, s, y, tol + 2.0 ** -149, 128, pow2)  # a denormal's step


@pytest.mark.parametrize("pow2", [False, True])
def test_power_of_two_borders(ws, pow2):
    """Group maxima at and beside 448 * 2^k: gamma sets y's magnitudes exactly (h = +-1, inv within 3 steps)."""
    N = 512
    parts = [torch.ones((1, N), dtype=torch.bfloat16, device="cuda")]
    gamma = torch.ones(N, device="cuda")
    for i, v in enumerate((448.0, 449.0, 447.0, 0.875, 0.8751, 2.0 ** -20, 1.75 * 2.0 ** 30, 1.0)):
        gamma[i * 64] = v
        gamma[i * 64 + 1:i * 64 + 64] = v / 3
    q, s, _ = run(ws, parts, None, gamma, 64, pow2)
    _, _, y, tol = ref.norm64(parts, None, gamma)
    ref.check_quant(q, s, y, tol, 64, pow2)


@pytest.mark.parametrize("pow2", [False, True])
def test_values_that_are_not_finite(ws, pow2):
    """A NaN or infinity takes its row's groups to NaN, other rows and finite groups stay."""
    parts, res, gamma = inputs(2, 5, 256, 3)
    parts[0][1, 7] = float("nan")
    parts[1][3, 200] = float("inf")
    q, s, _ = run(ws, parts, res, gamma, 128, pow2)
    nan = (s == 255) if pow2 else s.isnan()
    assert nan[1].all()                       # a NaN spoils the row's statistics
    assert not nan[3, 0] and nan[3, 1]        # inv = 0: the finite group is zero, inf * 0 is NaN
    assert (q[3, :128] & 0x7F == 0).all() and (q[3, 128:] == 0x7F).all() and (q[1] == 0x7F).all()
    keep = [0, 2, 4]
    _, _, y, tol = ref.norm64([p[keep] for p in parts], res[keep], gamma)
    ref.check_quant(q[keep], s[keep], y, tol, 128, pow2)


def test_in_place_residual_other_stream_and_guards(ws):
    """residual_out over residual, on a side stream; memory behind the last row stays."""
    parts, res, gamma = inputs(4, 9, 520, 11)
    q = torch.full((12, 520), 0x55, dtype=torch.uint8, device="cuda")
    s = torch.full((12, 17), 77.0, device="cuda")
    want = res.clone()
    q1, s1, r1 = run(ws, parts, res, gamma, 32, False)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    are.allreduce_rmsnorm_quant_groups(parts, want, gamma, ref.EPS, q[:9], s[:9], ws, group=32, residual_out=want,
                                       stream=st)
    torch.cuda.synchronize()
    assert torch.equal(q[:9], q1) and torch.equal(s[:9], s1) and torch.equal(want, r1)
    assert (q[9:] == 0x55).all() and (s[9:] == 77).all()


def test_graph_replays(ws):
    parts, res, gamma = inputs(8, 6, 7168, 21)
    q, s = outputs(6, 7168, 128, False)

    def call():
        are.allreduce_rmsnorm_quant_groups(parts, res, gamma, ref.EPS, q, s, ws)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(3):
        p2, r2, g2 = inputs(8, 6, 7168, 30 + k)
        for a, b in zip(parts + [res, gamma], p2 + [r2, g2]):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        _, _, y, tol = ref.norm64(parts, res, gamma)
        ref.check_quant(q, s, y, tol, 128, False)


def test_offsets_past_32_bits(ws):
    """More than 2^31 elements: the first and last rows."""
    M, N = (1 << 18) + 5, 8200
    x = torch.zeros((M, N), dtype=torch.bfloat16, device="cuda")
    rows = [0, 1, M // 2, M - 2, M - 1]
    parts, _, gamma = inputs(1, len(rows), N, 41, False)
    x[rows] = parts[0]
    q, s = outputs(M, N, 128, True)
    are.allreduce_rmsnorm_quant_groups([x], None, gamma, ref.EPS, q, s, ws)
    _, _, y, tol = ref.norm64(parts, None, gamma)
    ref.check_quant(q[rows], s[rows], y, tol, 128, True)
    assert (s[2] == 127).all() and (q[M - 3] == 0).all()


def test_refusals(ws):
    parts, res, gamma = inputs(2, 4, 256, 1)
    q, s = outputs(4, 256, 128, False)

    def call(parts=parts, res=res, gamma=gamma, q=q, s=s, **k):
        are.allreduce_rmsnorm_quant_groups(parts, res, gamma, k.pop("eps", ref.EPS), q, s, ws, **k)
    bad = [dict(group=96), dict(group=64), dict(q=q[:3]), dict(q=q.float()), dict(s=s.double()), dict(gamma=gamma[:128]),
           dict(parts=[]), dict(parts=parts * 5), dict(parts=[parts[0], parts[1].float()]), dict(res=res.t()),
           dict(parts=[parts[0].cpu(), parts[1]]), dict(parts=[p[:, ::2] for p in parts]), dict(residual_out=res[:2])]
    for k in bad:
        with pytest.raises(ValueError):
            call(**k)
    for k in (dict(eps=0.0), dict(eps=float("nan"))):
        with pytest.raises(are.AreError):
            call(**k)
    with pytest.raises(are.AreError):  # rows of 8 columns
        call([p[:, :36].contiguous() for p in parts], None, gamma[:36].contiguous(), q[:, :36].contiguous(), s[:, :1].contiguous())
    odd = torch.empty(4 * 256 + 8, dtype=torch.bfloat16, device="cuda")[4:4 + 1024].view(4, 256)
    with pytest.raises(are.AreError):  # 8 bytes off a 16-byte boundary
        call([odd, parts[1]])
    with are.Workspace(R_max=1, M_max=1, N_max=8) as small:
        with pytest.raises(are.AreError) as e:
            are.allreduce_rmsnorm_quant_groups(parts, res, gamma, ref.EPS, q, s, small)
        assert e.value.status == are.ECAPACITY
    empty = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    call([empty, empty], None, gamma, q[:0], s[:0])
    assert ws.last_launch()["kernel"] == "none"


@pytest.mark.parametrize("pow2", [False, True])
def test_magnitudes_over_all_of_fp32(ws, pow2):
    """Groups from below the smallest normal scale up to near fp32's largest value."""
    M, N = 6, 2048
    g = torch.Generator(device="cuda").manual_seed(17)
    sign = torch.randint(0, 2, (M, N), generator=g, device="cuda") * 2 - 1
    size = 2.0 ** -torch.randint(0, 3, (M, N), generator=g, device="cuda").double()
    parts = [(sign * size).to(torch.bfloat16)]
    e = torch.tensor([-140, -126, -118, -117, -116, -110, -60, -1, 0, 30, 100, 118, 119, 120, 121, 122, 123, 124, 125, 125,
                      -149, -130, -125, -119, 60, 119, 120, 120, 126, 126, 10, 90], device="cuda").double()
    gamma = (2.0 ** e * 0.9).repeat_interleave(64).float()
    q, s, ro = run(ws, parts, None, gamma, 64, pow2)
    _, _, y, tol = ref.norm64(parts, None, gamma)
    assert y.abs().max() < 3.4e38
    ref.check_quant(q, s, y, tol + 2.0 ** -149, 64, pow2)  # a denormal's step
