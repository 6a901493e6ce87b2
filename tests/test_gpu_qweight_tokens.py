"""8-bit tokens of the 4-bit linear at the ends of their scales' ranges, in every token tile."""
import pytest
import torch

import all_reduce_epilogue_gb300 as are
from tests import ops_ref as ref
from tests.test_gpu_qweight import tiled, weights  # noqa: F401 (a fixture)

pytestmark = pytest.mark.gpu


def value(xq, xs, xgroup):
    """The tokens in 64 bits; xs: E8M0 bytes or fp32."""
    f = ref.e8m0_value(xs) if xs.dtype == torch.uint8 else xs.double()
    return xq.view(torch.float8_e4m3fn).double() * f.repeat_interleave(xgroup, -1)[:, :xq.shape[1]]


def product(ws, xq, xs, w, group, xgroup):
    out = torch.full((xq[0].shape[0], w[0][0].shape[0]), 7.0, dtype=torch.bfloat16, device="cuda")
    are.gemm_ar_qweight_qx(xq, xs, [are.QWeight(*t, group) for t in w], out, ws, xgroup=xgroup)
    assert ws.device_status()["code"] == 0
    return out


def random_codes(g, *shape):
    q = torch.randint(0, 256, shape, generator=g, device="cuda", dtype=torch.uint8)
    q[(q & 0x7F) == 0x7F] = 0x38
    return q


@pytest.mark.parametrize("M", [3, 40])
def test_largest_power_of_two_scales(tiled, M):  # noqa: F811
    """Bytes 249 to 254: codes of zero, and codes of 1 under small weights, whose sums fp32 holds."""
    ws, _ = tiled
    R, N, K, group = 2, 40, 544, 128
    w, g = weights(R, N, K, group, True, 300 + M)
    for _, s, _ in w:
        s.mul_(2.0 ** -100)
    xq = [torch.zeros((M, K), dtype=torch.uint8, device="cuda") for _ in range(R)]
    xs = [torch.randint(249, 255, (M, 17), generator=g, device="cuda", dtype=torch.uint8) for _ in range(R)]
    xq[0][1:] = 0x38
    xq[1][2::3] = 0xB8
    out = product(ws, xq, xs, w, group, 32)
    assert (out[0] == 0).all()
    want, tol = ref.linear64([value(q, s, 32) for q, s in zip(xq, xs)], w, group)
    ref.check(out, want, tol, "out")


@pytest.mark.parametrize("odd", [0, 1])
def test_small_values_beside_a_large_one(tiled, odd):  # noqa: F811
    """One value of 448 * 2^-d, d = 18 to 100, at an even or an odd k, beside one of 448 whose weights are zero: exact."""
    ws, _ = tiled
    N, K, group = 72, 256, 32
    w, _ = weights(1, N, K, group, False, 310)
    w[0][0][:, 0] = 0x88  # k = 0 and 1 weigh nothing
    d = torch.cat((torch.arange(18, 36), torch.arange(40, 101, 10))).cuda()
    M = len(d)
    xq = torch.zeros((M, K), dtype=torch.uint8, device="cuda")
    xs = torch.full((M, 8), 127, dtype=torch.uint8, device="cuda")
    xq[:, 0] = 0x7E
    at = 32 + 2 * torch.arange(M, device="cuda") * 4 + odd  # in groups 1 to 7
    xq[torch.arange(M, device="cuda"), at] = 0x7E
    xs[torch.arange(M, device="cuda"), at // 32] = (127 - d).to(torch.uint8)
    out = product(ws, [xq], [xs], w, group, 32)
    want, tol = ref.linear64([value(xq, xs, 32)], w, group)
    ref.check(out, want, tol - 1e-38, "out")


@pytest.mark.parametrize("K,xgroup", [(256, 32), (544, 32), (512, 128)])
def test_groups_of_zeros_beside_small_ones(tiled, K, xgroup):  # noqa: F811
    """In every 256 k a group of zeros, under the scale 1 that the quantised norm gives it or the largest there is; the
    others' scales are 2^-20 to 2^-40, the same in a row, so that what a row loses shows in its own sums."""
    ws, _ = tiled
    R, M, N, group = 2, 41, 72, 128
    w, g = weights(R, N, K, group, True, 320 + K)
    G = -(-K // xgroup)
    byte = 87 + torch.arange(M, device="cuda") // 2
    xq, xs = [], []
    for r in range(R):
        q = random_codes(g, M, K)
        s = byte[:, None].repeat(1, G).to(torch.uint8)
        for a in range(r % 2, G, 256 // xgroup):
            q[:, a * xgroup:(a + 1) * xgroup] = 0
            s[0::2, a], s[1::2, a] = 127, 254
        xq.append(q), xs.append(s)
    xq[0][5], xq[1][5] = 0, 0  # and a token of zeros
    out = product(ws, xq, xs, w, group, xgroup)
    want, tol = ref.linear64([value(q, s, xgroup) for q, s in zip(xq, xs)], w, group)
    ref.check(out, want, tol, "out")
    assert (out[5] == 0).all()


@pytest.mark.parametrize("xgroup", [32, 128])
def test_small_fp32_scales(tiled, xgroup):  # noqa: F811
    """fp32 token scales from 2^-126 to 2^-90, a magnitude a token; outputs down to bf16's smallest.  The sums are kept
    2^17 smaller than the output, where a step of fp32 is 2^-149 at least: half a step for a product of scales, times up
    to 2^2.7 (the sum that it multiplies), and one for the sum, a group: 2^17 * 2^-150 * 8."""
    ws, _ = tiled
    R, M, N, K, group = 2, 37, 72, 544, 128
    w, g = weights(R, N, K, group, True, 330 + xgroup)
    G = -(-K // xgroup)
    e = torch.arange(M, device="cuda") - 126.0
    xq = [random_codes(g, M, K) for _ in range(R)]
    xs = [torch.exp2(e)[:, None] * (1 + torch.rand((M, G), generator=g, device="cuda")) for _ in range(R)]
    out = product(ws, xq, xs, w, group, xgroup)
    want, tol = ref.linear64([value(q, s, xgroup) for q, s in zip(xq, xs)], w, group)
    ref.check(out, want, tol + R * max(G, -(-K // group)) * 2.0 ** -130 + 2.0 ** -134, "out")


@pytest.mark.parametrize("M", [2, 40])
def test_bf16_tokens_below_the_normal_ones(tiled, M):  # noqa: F811
    """Tokens that are all subnormal, under weights large enough for normal outputs; and subnormal beside normal ones."""
    ws, _ = tiled
    R, N, K, group = 2, 72, 544, 64
    w, g = weights(R, N, K, group, True, 350 + M)
    for _, s, _ in w:
        s.mul_(2.0 ** 30)
    x = []
    for _ in range(R):
        bits = torch.randint(1, 128, (M, K), generator=g, device="cuda", dtype=torch.int16)
        x.append(torch.where(torch.rand((M, K), generator=g, device="cuda") < 0.5, bits, bits - 32768).view(torch.bfloat16))
    x[0][1, 300:] = (torch.randn(K - 300, generator=g, device="cuda") * 2.0 ** -120).to(torch.bfloat16)
    x[1][0, :256] = 0
    out = torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda")
    are.gemm_ar_qweight(x, [are.QWeight(*t, group) for t in w], out, ws)
    assert ws.device_status()["code"] == 0
    want, tol = ref.linear64(x, w, group)
    ref.check(out, want, tol - 1e-38, "out")


@pytest.mark.parametrize("K,group", [(32, 32), (128, 128)])
def test_small_tokens_beside_one_that_weighs_nothing(tiled, K, group):  # noqa: F811
    """A token of 1 under codes equal to their zero points, among ones of 2^-12.  What is cut of 16 products and the sum
    so far: 2^-18 each in the one instruction that has the large token, and 2^-25 of the sum so far, below 2^4, in those
    that go on from it.  The zero point's product and the difference are of magnitude 15 * (1 + K * 2^-12): a sum of
    tokens takes up to 10 additions, the rest 2."""
    ws, _ = tiled
    M, N = max(K, 64), 64
    g = torch.Generator(device="cuda").manual_seed(360 + K)
    u = torch.randint(1, 16, (N, K), generator=g, device="cuda", dtype=torch.uint8)
    zero = torch.randint(1, 16, (N, 1), generator=g, device="cuda", dtype=torch.uint8)
    x = (2.0 ** -12 * (0.5 + 0.5 * torch.rand((M, K), generator=g, device="cuda"))).to(torch.bfloat16)
    at = torch.arange(M, device="cuda") % K
    x[torch.arange(M, device="cuda"), at] = 1
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    one = torch.ones((N, 1), dtype=torch.bfloat16, device="cuda")
    for m in range(0, M, max(1, M // 16)):
        v = u.clone()
        v[:, at[m]] = zero[:, 0]
        codes = (v[:, 0::2] | v[:, 1::2] << 4).contiguous()
        are.gemm_ar_qweight([x], [are.QWeight(codes, one, zero, group)], out, ws)
        want = x[m].double() @ (v.double() - zero.double()).T
        magnitude = 15 * (1 + K * 2.0 ** -12)
        tol = 17 * 2.0 ** -18 + (K // 16 - 1) * 17 * 2.0 ** -21 + 12 * ref.U * magnitude
        ref.check(out[m], want, tol + ref.BF16 * (want.abs() + tol), f"token {m}")
