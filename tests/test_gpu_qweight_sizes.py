"""The largest sizes of the 4-bit linear."""
import pytest
import torch

import all_reduce_epilogue_gb300 as are
from tests import ops_ref as ref
from tests.gpu_util import need_gpu
from tests.test_gpu_qweight import tokens8, weights

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    need_gpu()
    with are.Workspace(R_max=8, M_max=1, N_max=8) as w:
        yield w


# the longest rows; rows as long as the staging buffer of eight ranks takes for one
@pytest.mark.parametrize("R,M,N,K", [(1, 1, 40, 1 << 20), (8, 2, 8, 1 << 20), (1, 9, 16, 1 << 20), (1, 20, 40, 400000),
                                     (1, 33, 264, 200032), (2, 17, 8, 131104)])
@pytest.mark.parametrize("kind", ["bf16", "fp32", "e8m0"])
def test_long_rows(ws, R, M, N, K, kind):
    w, g = weights(R, N, K, 32, True, K + M)
    x = [torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16) for _ in range(R)]
    qw, out = [are.QWeight(*t, 32) for t in w], torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    vals = x
    if kind == "bf16":
        are.gemm_ar_qweight(x, qw, out, ws)
    else:
        t = [tokens8(v.float(), 128, kind == "e8m0") for v in x]
        are.gemm_ar_qweight_qx([v[0] for v in t], [v[1] for v in t], qw, out, ws, xgroup=128)
        vals = [v[2] for v in t]
    assert ws.device_status()["code"] == 0
    want, tol = ref.linear64(vals, w, 32)
    ref.check(out, want, tol, "out")


@pytest.mark.parametrize("M,variant", [(20, 2), (20, 4)])
def test_staged_tiles_of_more_than_2_32_weights(M, variant):
    """The first and the last rows."""
    need_gpu()
    N, K = (1 << 19) + 40, 8224
    codes = torch.zeros((N, K // 2), dtype=torch.uint8, device="cuda")
    scale = torch.ones((N, 257), dtype=torch.bfloat16, device="cuda")
    w, g = weights(1, 80, K, 32, False, 8)
    for a, b in ((0, 40), (N - 40, N)):
        codes[a:b], scale[a:b] = w[0][0][-(b - a):], w[0][1][-(b - a):]
    x = [torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)]
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    with are.Workspace(R_max=8, M_max=1, N_max=8) as ws:
        ws.set_debug(are.DEBUG_QWEIGHT_STAGED, 8 * variant)
        are.gemm_ar_qweight(x, [are.QWeight(codes, scale, None, 32)], out, ws)
        assert ws.device_status()["code"] == 0 and ws.last_launch()["variant"] == variant
    want, tol = ref.linear64(x, [(w[0][0][-40:], w[0][1][-40:], None)], 32)
    ref.check(out[:, :40], want, tol, "first rows")
    ref.check(out[:, -40:], want, tol, "last rows")
