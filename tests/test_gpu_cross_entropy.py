"""Softmax cross entropy of an output layer split over the ranks, and its gradients."""
import ctypes

import pytest
import torch

import all_reduce_epilogue_gb300 as are
from tests import ends_ref as ref
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    need_gpu()
    with are.Workspace(R_max=8, M_max=1100, N_max=8, K_max=1024, vocab_piece=1024) as w:
        yield w


def inputs(R, M, N, K, seed, vocab=None, wide=True, spread=1.5):
    g = torch.Generator(device="cuda").manual_seed(seed)
    vocab = R * N if vocab is None else vocab
    w = [(torch.randn((N, K), generator=g, device="cuda") * (spread / K ** 0.5)).to(torch.bfloat16) for _ in range(R)]
    t = torch.randint(0, vocab, (M,), generator=g, device="cuda")
    h = torch.randn((M, K), generator=g, device="cuda")
    h[::2] += 4 * torch.cat(w)[t[::2]].float()   # tokens that are foreseen
    if M > 3:
        t[3], t[1] = -100, vocab                 # no target: below and above the vocabulary
    if M > 5:
        t[5] = vocab - 1
    dloss = (0.5 + torch.rand(M, generator=g, device="cuda")) / max(M, 1)
    return h.to(torch.bfloat16), w, t if wide else t.int(), dloss


def run(ws, h, w, t, dloss, vocab=None, dh=True, dw=True, stream=None):
    (M, K), N = h.shape, w[0].shape[0]
    loss, lse = (torch.full((M,), 7.0, device="cuda") for _ in range(2))
    are.gemm_cross_entropy(h, w, t, loss, lse, ws, vocab=vocab, stream=stream)
    gh = torch.full((M, K), 7.0, dtype=torch.bfloat16, device="cuda") if dh else None
    gw = torch.full((len(w), N, K), 7.0, dtype=torch.bfloat16, device="cuda") if dw else None
    are.gemm_cross_entropy_backward(h, w, t, lse, dloss, gh, list(gw) if dw else None, ws, vocab=vocab, stream=stream)
    assert ws.device_status()["code"] == 0, ws.device_status()
    return loss, lse, gh, gw


def compare(got, want):
    for g, (v, tol), what in zip(got, want, ("loss", "lse", "dh", "dw")):
        ref.check(g, v, tol, what)


# one token and one column; part of a tile, one tile, tiles on both sides of 128 and 256; ranks shorter and longer than a
# tile; K below, at and past a block of 64; several pieces (1024 columns at 1100 rows); split sums (few rows)
SHAPES = [(1, 1, 1, 8), (1, 1, 256, 64), (1, 128, 256, 64), (2, 5, 100, 72), (1, 256, 256, 256), (3, 77, 367, 200),
          (8, 1, 333, 1024), (1, 300, 1000, 136), (4, 129, 511, 520), (1, 1, 30000, 64), (2, 64, 5000, 256), (8, 257, 40, 1000),
          (1, 1100, 5000, 128), (3, 1025, 1537, 264), (5, 600, 1300, 1024), (1, 20, 70000, 512),
          (1, 8, 3000, 64), (2, 9, 700, 72), (3, 16, 240, 128), (2, 17, 1000, 136), (1, 31, 241, 64), (4, 33, 600, 200),
          (1, 96, 40000, 64), (7, 127, 321, 96), (2, 128, 2000, 1024), (1, 3, 111000, 8)]


@pytest.mark.parametrize("R,M,N,K", SHAPES)
def test_against_64_bits(ws, R, M, N, K):
    h, w, t, dloss = inputs(R, M, N, K, R + M + N + K)
    got = run(ws, h, w, t, dloss)
    compare(got, ref.cross_entropy64(h, w, t, R * N, dloss))
    last = ws.last_launch()
    assert last["kernel"] == "xent_kernel<DLogits>" and (last["cluster"], last["block"]) == ((1, 256) if M <= 128 else (2, 640))
    for a, b in zip(got, run(ws, h, w, t.int(), dloss)):   # the same bits again, and from 32-bit targets
        assert torch.equal(a, b)
    assert torch.equal(run(ws, h, w, t, dloss, dw=False)[2], got[2])
    assert torch.equal(run(ws, h, w, t, dloss, dh=False)[3], got[3])


@pytest.mark.parametrize("R,N,vocab", [(3, 367, 1100), (4, 256, 769), (2, 300, 300), (8, 100, 150), (1, 512, 1), (3, 400, 401),
                                       (4, 1000, 1200), (2, 700, 1)])
def test_padded_vocabulary(ws, R, N, vocab):
    """Weights behind the vocabulary take no part, whatever they hold; their gradients are zero."""
    for M in (70, 300):
        h, w, t, dloss = inputs(R, M, N, 96, vocab, vocab=vocab)
        full = torch.cat(w)
        full[vocab:] = float("nan")
        full[vocab + 1::2] = float("inf")
        w = list(full.view(R, N, -1).clone())
        got = run(ws, h, w, t, dloss, vocab=vocab)
        compare(got, ref.cross_entropy64(h, w, t, vocab, dloss))
        assert (got[3].flatten(0, 1)[vocab:] == 0).all()
        assert torch.equal(run(ws, h, w, t, dloss, vocab=vocab, dh=False)[3], got[3])


def test_foreseen_tokens_and_large_logits(ws):
    """Losses near zero keep their relative accuracy as far as the logits have it; logits of +-300 neither overflow nor
    vanish."""
    h, w, t, dloss = inputs(2, 40, 700, 256, 5, spread=8.0)
    h = (h.float() * 8).to(torch.bfloat16)
    got = run(ws, h, w, t, dloss)
    compare(got, ref.cross_entropy64(h, w, t, 1400, dloss))
    # one column far above the rest by an exact amount: loss = log(1 + 1399 exp(-16)) from logits that are exact
    h = torch.zeros((4, 64), dtype=torch.bfloat16, device="cuda")
    h[:, 0] = 16
    w = [torch.zeros((700, 64), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    w[1][17, 0] = 1
    t = torch.full((4,), 717, device="cuda")
    loss, lse, dh, dw = run(ws, h, w, t, dloss[:4])
    want = torch.log1p(1399 * torch.exp(torch.tensor(-16.0, dtype=torch.float64))).item()
    assert abs(loss[0].item() / want - 1) < 2e-3    # log(1 + 1.6e-4) in fp32: 2^-24 of 1 under 1.6e-4, and exp's 2^-22
    p = 1 / (1 + 1399 * torch.exp(torch.tensor(-16.0, dtype=torch.float64))).item()
    g = (p - 1) * dloss[:4].double()
    # g (p - 1) from expm1(z - lse), whose error is lse's rounding, 2^-24 * 16 against 1.6e-4
    ref.check(dh[:, 0], g, g.abs() * (2.0 ** -7 + 1e-2), "dh")


def test_rows_without_a_target_and_nan(ws):
    """A row whose hidden state is NaN has NaN results and leaves the others alone; without a target its gradient is 0."""
    h, w, t, dloss = inputs(2, 9, 300, 128, 3)
    bad = h.clone()
    bad[3, 5] = float("nan")     # row 3 has no target
    bad[6, 7] = float("inf")
    keep = [0, 1, 2, 4, 5, 7, 8]
    got = run(ws, bad, w, t, dloss, dw=False)
    want = ref.cross_entropy64(h[keep], w, t[keep], 600, dloss[keep])
    compare([g[keep] if g is not None else None for g in got[:3]], want[:3])
    assert got[1][3].isnan() and not got[0][6].isfinite() and not got[1][6].isfinite() and (got[2][3] == 0).all()
    assert got[0][3] == 0
    # rows without a target (1 and 3) take no part in dw, whatever they hold
    for M in (9, 200):
        h2, w2, t2, g2 = inputs(2, M, 300, 128, 13)
        wild = h2.clone()
        wild[3], wild[1, ::2] = float("nan"), float("inf")
        _, _, dh, dw = run(ws, wild, w2, t2, g2)
        want = ref.cross_entropy64(h2, w2, t2, 600, g2)
        ref.check(dh, *want[2], "dh")
        ref.check(dw, *want[3], "dw")
    # no row has a target
    none = torch.full((9,), -100, device="cuda")
    loss, _, dh, dw = run(ws, h, w, none, dloss)
    assert (loss == 0).all() and (dh == 0).all() and (dw == 0).all()


def test_against_differences(ws):
    """sum(dloss * loss) by central differences of the 64-bit formula, in random directions."""
    h, w, t, dloss = inputs(2, 12, 90, 64, 21)
    _, _, dh, dw = run(ws, h, w, t, dloss)
    want = ref.cross_entropy64(h, w, t, 180, dloss)
    g = torch.Generator(device="cuda").manual_seed(4)

    def total(x, y):
        z = x @ y.T
        on = (t >= 0) & (t < 180)
        return (torch.where(on, torch.logsumexp(z, 1) - z.gather(1, t.clamp(0, 179)[:, None])[:, 0], 0.0) * dloss.double()).sum()
    x, y, step = h.double(), torch.cat(w).double(), 1e-5
    for _ in range(5):
        a, b = torch.randn(x.shape, generator=g, device="cuda").double(), torch.randn(y.shape, generator=g, device="cuda").double()
        num = (total(x + step * a, y) - total(x - step * a, y)) / (2 * step)
        assert abs(num - (dh.double() * a).sum()) <= (want[2][1] * a.abs()).sum() + 1e-8
        num = (total(x, y + step * b) - total(x, y - step * b)) / (2 * step)
        assert abs(num - (dw.double().flatten(0, 1) * b).sum()) <= (want[3][1].flatten(0, 1) * b.abs()).sum() + 1e-8


def test_pieces_give_the_same_loss_and_close_gradients(ws):
    """The smallest workspace, whose buffer holds 8 tiles of d backward, 131 tiles' pairs forward (few tokens: 163 and 10485):
    several pieces both ways, the last one short."""
    for M, N, K in ((1000, 12001, 64), (50, 23100, 8), (128, 181000, 8)):
        h, w, t, dloss = inputs(3, M, N, K, 8)
        with are.Workspace(R_max=3, M_max=M, N_max=8, K_max=K, vocab_piece=1) as small:
            got = run(small, h, w, t, dloss)
        compare(got, ref.cross_entropy64(h, w, t, 3 * N, dloss))


def test_guards_stream_and_no_rows(ws):
    h, w, t, dloss = inputs(2, 33, 301, 72, 2)
    loss, lse = (torch.full((40,), 9.0, device="cuda") for _ in range(2))
    dh = torch.full((36, 72), 3.0, dtype=torch.bfloat16, device="cuda")
    dw = torch.full((2, 304, 72), 3.0, dtype=torch.bfloat16, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    are.gemm_cross_entropy(h, w, t, loss[:33], lse[:33], ws, stream=s)
    are.gemm_cross_entropy_backward(h, w, t, lse[:33], dloss, dh[:33], [dw[0, :301], dw[1, :301]], ws, stream=s)
    torch.cuda.synchronize()
    compare((loss[:33], lse[:33], dh[:33], dw[:, :301]), ref.cross_entropy64(h, w, t, 602, dloss))
    assert (loss[33:] == 9).all() and (lse[33:] == 9).all() and (dh[33:] == 3).all() and (dw[:, 301:] == 3).all()
    loss, lse, dh, dw = run(ws, h[:0], w, t[:0], dloss[:0])
    assert loss.shape == (0,) and (dw == 0).all()


def test_graph_replays(ws):
    R, M, N, K = 2, 200, 900, 128
    h, w, t, dloss = inputs(R, M, N, K, 1)
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty((R, N, K), dtype=torch.bfloat16, device="cuda")

    def call():
        are.gemm_cross_entropy(h, w, t, loss, lse, ws)
        are.gemm_cross_entropy_backward(h, w, t, lse, dloss, dh, list(dw), ws)
    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for k in range(3):
        h2, w2, t2, d2 = inputs(R, M, N, K, 50 + k)
        for a, b in zip([h, t, dloss, *w], [h2, t2, d2, *w2]):
            a.copy_(b)
        g.replay()
        torch.cuda.synchronize()
        compare((loss, lse, dh, dw), ref.cross_entropy64(h, w, t, R * N, dloss))


def test_offsets_past_32_bits():
    """Weights and their gradients of more than 2^32 bytes in one rank."""
    need_gpu()
    M, N, K = 3, (1 << 22) + 300, 520
    h, w, t, dloss = inputs(1, M, 64, K, 9)
    big = torch.zeros((N, K), dtype=torch.bfloat16, device="cuda")
    rows = torch.cat([torch.arange(32), torch.arange(N - 32, N)]).cuda()
    big[rows] = w[0]
    t = rows[t]
    with are.Workspace(R_max=1, M_max=4, N_max=8, K_max=K, vocab_piece=1 << 20) as ws:
        dw = torch.empty_like(big)
        loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        are.gemm_cross_entropy(h, [big], t, loss, lse, ws)
        dh = torch.empty_like(h)
        are.gemm_cross_entropy_backward(h, [big], t, lse, dloss, dh, [dw], ws)
        assert ws.device_status()["code"] == 0
    z = h.double() @ w[0].double().T
    want = torch.log(torch.exp(z).sum(1) + (N - 64))
    ref.check(lse, want, 1e-5 * want.abs(), "lse")
    p = torch.exp(z - want[:, None])
    hot = torch.zeros_like(p)
    hot[torch.arange(M), (rows[None] == t[:, None]).int().argmax(1)] = 1
    d = (p - hot) * dloss.double()[:, None]
    ref.check(dw[rows], d.T @ h.double(), 2.0 ** -6 * (d.abs().T @ h.double().abs()) + 1e-7, "dw")
    ref.check(dh, d @ w[0].double(), 2.0 ** -6 * (d.abs() @ w[0].double().abs()) + 1e-7, "dh")


def test_refusals(ws):
    h, w, t, dloss = inputs(2, 6, 80, 64, 1)
    loss, lse = torch.empty(6, device="cuda"), torch.empty(6, device="cuda")
    dh, dw = torch.empty_like(h), [torch.empty_like(x) for x in w]
    for kw in (dict(h=h.float()), dict(h=h[:, :32]), dict(w=[w[0], w[1][:40]]), dict(w=[]), dict(t=t[:5]), dict(t=t.float()),
               dict(t=t.cpu()), dict(loss=loss[:5]), dict(lse=lse.double()), dict(vocab=0), dict(vocab=161), dict(w=[w[0].cpu()] * 2)):
        a = dict(h=h, w=w, t=t, loss=loss, lse=lse, vocab=None)
        a.update(kw)
        with pytest.raises(ValueError):
            are.gemm_cross_entropy(a["h"], a["w"], a["t"], a["loss"], a["lse"], ws, vocab=a["vocab"])
    for kw in (dict(dh=dh[:5]), dict(dw=dw[:1]), dict(dloss=dloss.double()), dict(dw=[dw[0], dw[1].float()])):
        a = dict(dh=dh, dw=dw, dloss=dloss)
        a.update(kw)
        with pytest.raises(ValueError):
            are.gemm_cross_entropy_backward(h, w, t, lse, a["dloss"], a["dh"], a["dw"], ws)
    for kw in (dict(dw=[dw[0], dw[0]]), dict(dw=[dw[0], w[1]]), dict(dh=h), dict(dh=dw[1][:6])):   # overlapping outputs
        a = dict(dh=dh, dw=dw)
        a.update(kw)
        with pytest.raises(are.AreError) as e:
            are.gemm_cross_entropy_backward(h, w, t, lse, dloss, a["dh"], a["dw"], ws)
        assert e.value.status == are.EINVAL
    with pytest.raises(are.AreError):
        are.gemm_cross_entropy(h, w, t, loss, loss, ws)
    odd = torch.empty((6, 60), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(are.AreError):
        are.gemm_cross_entropy(odd, [odd], t, loss, lse, ws)      # K % 8
    for caps in (dict(vocab_piece=0), dict(R_max=1), dict(M_max=5), dict(K_max=32)):
        c = dict(R_max=2, M_max=8, N_max=8, K_max=64, vocab_piece=256)
        c.update(caps)
        with are.Workspace(**c) as other:
            with pytest.raises(are.AreError) as e:
                are.gemm_cross_entropy(h, w, t, loss, lse, other)
            assert e.value.status == are.ECAPACITY
    with pytest.raises(are.AreError):
        are.Workspace(R_max=1, M_max=1, N_max=8, vocab_piece=256)   # K_max missing


@pytest.mark.parametrize("M,K_max", [(77, 1001), (1, 1001), (5, 1002), (131, 1004)])
def test_capacities_that_are_no_multiple_of_8(M, K_max):
    """Workspaces take any K_max: both directions, in several pieces of the smallest buffer."""
    need_gpu()
    R, N, K = 3, 14000 if M > 5 else 12, 1000
    h, w, t, dloss = inputs(R, M, N, K, K_max)
    want = ref.cross_entropy64(h, w, t, R * N, dloss)
    with are.Workspace(R_max=R, M_max=M, N_max=8, K_max=K_max, vocab_piece=1) as ws:
        got = run(ws, h, w, t, dloss)
        compare(got, want)
        assert torch.equal(run(ws, h, w, t, dloss, dw=False)[2], got[2])


def test_capacities_that_no_device_holds():
    need_gpu()
    with pytest.raises(are.AreError) as e:
        are.Workspace(R_max=1, M_max=1, N_max=8, K_max=(1 << 63) - 8, vocab_piece=256)
    assert e.value.status == are.ENOMEM


def half_step(v):
    """Half a step of bf16 at |v|."""
    return torch.ldexp(torch.ones_like(v), torch.frexp(v.abs())[1] - 9)


def gradient_bounds(h, w, t, vocab, dloss):
    """dh, dw in 64 bits, each with the bound of products of an fp32 d, rounded to bf16 once: as ref.cross_entropy64, with
    2^-16 for d's two bf16 parts (half a step of bf16 of what half a step of bf16 left) in place of a half step, twice the
    terms for the two parts, and the result's own half step."""
    K, x, y = h.shape[1], h.double(), torch.cat([v.double() for v in w])[:vocab]
    U = 2.0 ** -24
    z = x @ y.T
    err = (min(K / 16, 64) + K / 512 + 16) * 2 * U * (x.abs() @ y.abs().T)
    lse = torch.logsumexp(z, 1, keepdim=True)
    tol_lse = err.max(1, keepdim=True).values + 2.0 ** -20 + 2 * U * lse.abs()
    on = ((t >= 0) & (t < vocab))[:, None]
    g = torch.where(on, dloss.double()[:, None], 0.0)
    p = torch.exp(z - lse)
    d = (p - torch.zeros_like(p).scatter_(1, t.long().clamp(0, vocab - 1)[:, None], 1.0)) * g
    e = p * g * (err + tol_lse + 2.0 ** -20) * 1.1
    e = e + 2.0 ** -16 * (d.abs() + e)
    out = []
    for a, ea, b, n in ((d, e, y, vocab), (d.T, e.T, x, len(h))):
        want = a @ b
        tol = ea @ b.abs() + (n / 8 + 64) * 2 * U * (a.abs() @ b.abs())
        out.append((want, tol + half_step(want.abs() + tol) + 1e-30))
    return out


@pytest.mark.parametrize("R,M,N,K", [(2, 40, 90, 64), (1, 128, 300, 64), (3, 200, 70, 64), (1, 600, 500, 72), (2, 3, 700, 8)])
def test_gradients_are_as_near_as_fp32_products(ws, R, M, N, K):
    h, w, t, dloss = inputs(R, M, N, K, 7 * M + K)
    want = gradient_bounds(h, w, t, R * N, dloss)
    _, _, dh, dw = run(ws, h, w, t, dloss)
    ref.check(dh, *want[0], "dh")
    ref.check(dw.flatten(0, 1), *want[1], "dw")


def test_one_part_of_the_logits_gradient(ws):
    """A caller may have the logits' gradient rounded to bf16 once: within a half step of each term, and not within 2^-16."""
    for M in (40, 300):
        h, w, t, dloss = inputs(2, M, 500, 64, M)
        loss, lse, dh, dw = run(ws, h, w, t, dloss)
        ws.set_logit_gradient(1)
        try:
            got = run(ws, h, w, t, dloss)
            again = run(ws, h, w, t, dloss, dw=False)[2]
        finally:
            ws.set_logit_gradient(2)
        compare(got, ref.cross_entropy64(h, w, t, 1000, dloss))
        assert torch.equal(got[0], loss) and torch.equal(got[1], lse) and torch.equal(again, got[2])
        far = [((g.double().view_as(v) - v).abs() > tol).any() for g, (v, tol) in zip(got[2:], gradient_bounds(h, w, t, 1000, dloss))]
        assert all(far)
        back = run(ws, h, w, t, dloss)
        assert torch.equal(back[2], dh) and torch.equal(back[3], dw)
    for parts in (0, 3, -1):
        with pytest.raises(are.AreError):
            ws.set_logit_gradient(parts)


def test_the_reserved_word_of_the_capacities_is_not_read():
    """A caller from before the cross entropy may have left it unset: the workspace is made, without the cross entropy's
    buffers."""
    need_gpu()
    lib = are.load_library()
    free = []
    for word in (0, 0xDEADBEEF, 4096, 1 << 28):
        for K_max in (0, 512):
            caps, ws = are._Caps(2, 65536, 64, K_max, 0, 0, word), ctypes.c_void_p()
            assert lib.are_workspace_create(ctypes.byref(ws), ctypes.byref(caps)) == are.OK
            if K_max:
                free.append(torch.cuda.mem_get_info()[0])
            assert lib.are_workspace_destroy(ws) == are.OK
    assert max(free) - min(free) < 1 << 26   # (4096 columns of 65536 rows are 2^30 bytes)


def test_buffers_made_changed_and_released():
    need_gpu()
    h, w, t, dloss = inputs(2, 60, 3000, 64, 1)
    want = ref.cross_entropy64(h, w, t, 6000, dloss)
    with are.Workspace(R_max=2, M_max=60, N_max=8, K_max=64) as ws:
        for columns in (0, 256, 5000, 256, 0):
            ws.set_vocab_piece(columns)
            if columns:
                compare(run(ws, h, w, t, dloss), want)
            else:
                with pytest.raises(are.AreError) as e:
                    run(ws, h, w, t, dloss)
                assert e.value.status == are.ECAPACITY
        ws.set_vocab_piece(256)
        for columns in (-1, (1 << 28) + 1):
            with pytest.raises(are.AreError) as e:
                ws.set_vocab_piece(columns)
            assert e.value.status == are.EINVAL
        compare(run(ws, h, w, t, dloss), want)
    with are.Workspace(R_max=2, M_max=60, N_max=8) as ws, pytest.raises(are.AreError):
        ws.set_vocab_piece(256)   # K_max missing


@pytest.mark.parametrize("M", [9, 200, 1000])
def test_zeros_whatever_the_other_operand_holds(ws, M):
    """Rows without a target have dh 0 whatever the weights hold, padding has dw 0 whatever the hidden states do."""
    R, N, K, vocab = 3, 401, 96, 1100
    h, w, t, dloss = inputs(R, M, N, K, M, vocab=vocab)
    none = (t < 0) | (t >= vocab)
    bad = [v.clone() for v in w]
    bad[0][5, 3], bad[1][400, 7] = float("inf"), float("nan")
    dh = run(ws, h, bad, t, dloss, vocab=vocab)[2]
    assert none.any() and (dh[none] == 0).all() and dh[~none].isnan().any()
    wild = h.clone()
    wild[5, 3], wild[6, 9] = float("inf"), float("nan")    # both have a target
    _, _, dh, dw = run(ws, wild, w, t, dloss, vocab=vocab)
    dw = dw.flatten(0, 1)
    assert (dw[vocab:] == 0).all() and dw[:vocab].isnan().any() and (dh[none] == 0).all()
    with are.Workspace(R_max=R, M_max=M, N_max=8, K_max=K, vocab_piece=1) as small:   # (1000 rows: fp32 sums over pieces)
        assert (run(small, h, bad, t, dloss, vocab=vocab)[2][none] == 0).all()


@pytest.mark.parametrize("M", [40, 300])
def test_graph_replays_of_a_padded_vocabulary(ws, M):
    """Zeros for whole ranks behind the vocabulary stand before the kernels; several pieces, both numbers of parts."""
    R, N, K, vocab = 4, 2100, 64, 5000
    h, w, t, dloss = inputs(R, M, N, K, M, vocab=vocab)
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    dh, dw = torch.empty_like(h), torch.empty((R, N, K), dtype=torch.bfloat16, device="cuda")
    run(ws, h, w, t, dloss, vocab=vocab)
    graphs = []
    for parts in (1, 2):
        ws.set_logit_gradient(parts)
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            are.gemm_cross_entropy(h, w, t, loss, lse, ws, vocab=vocab)
            are.gemm_cross_entropy_backward(h, w, t, lse, dloss, dh, list(dw), ws, vocab=vocab)
    for k in range(4):
        h2, w2, t2, d2 = inputs(R, M, N, K, 60 + k, vocab=vocab)
        for a, b in zip([h, t, dloss, *w], [h2, t2, d2, *w2]):
            a.copy_(b)
        dw.fill_(5)
        graphs[k % 2].replay()
        torch.cuda.synchronize()
        compare((loss, lse, dh, dw), ref.cross_entropy64(h, w, t, vocab, dloss))
        assert (dw.flatten(0, 1)[vocab:] == 0).all()
        if k % 2:
            eager = run(ws, h, w, t, dloss, vocab=vocab)
            assert torch.equal(eager[2], dh) and torch.equal(eager[3], dw)
