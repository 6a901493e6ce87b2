"""Lookup in a table split over the ranks, and its gradient by sorted tokens."""
import pytest
import torch

import all_reduce_epilogue_gb300 as are
from tests.ends_ref import BF16, U, check
from tests.gpu_util import need_gpu

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ws():
    need_gpu()
    with are.Workspace(R_max=8, M_max=70000, N_max=8192) as w:
        yield w


def rand(seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16), g


def tokens(kind, M, V, g):
    if kind == "uniform":
        ids = torch.randint(0, V, (M,), generator=g, device="cuda")
    elif kind == "one":         # a single id: one sum over everything
        ids = torch.full((M,), V - 1, device="cuda")
    elif kind == "runs":        # every id a few times in a row, ends of chunks within them
        ids = (torch.arange(M, device="cuda") // 5) % V
    else:                       # text: a few ids make up much of it, some positions hold none
        u = torch.rand(M, generator=g, device="cuda", dtype=torch.float64)
        ids = (torch.exp(u * torch.log(torch.tensor(V + 1.0, dtype=torch.float64))).long() - 1).clamp(0, V - 1)
        ids[torch.rand(M, generator=g, device="cuda") < 0.1] = -1
        ids[M // 2] = V         # behind the vocabulary
    return ids


@pytest.mark.parametrize("R,M,N,V", [(1, 1, 8, 1), (2, 5, 2048, 160), (3, 7, 1032, 367), (8, 100, 64, 50), (4, 1000, 8192, 33),
                                     (1, 513, 4104, 1000), (2, 3, 32768, 5), (5, 3000, 24, 7)])
def test_lookup(ws, R, M, N, V):
    r, g = rand(R + M + N + V)
    tables = [r(V, N) for _ in range(R)]
    ids = tokens("text", M, R * V, g)
    full = torch.cat(tables)
    inside = (ids >= 0) & (ids < R * V)
    rows = torch.where(inside[:, None], full[ids.clamp(0, R * V - 1)], 0.0).to(torch.bfloat16)
    for wide in (True, False):
        buf = torch.full((M + 2, N), 9.0, dtype=torch.bfloat16, device="cuda")
        are.embedding_ar(ids if wide else ids.int(), tables, buf[:M], ws)
        assert torch.equal(buf[:M], rows) and (buf[M:] == 9).all()
        are.embedding_ar(ids if wide else ids.int(), tables, buf[:M], ws, scale=0.3)
        assert torch.equal(buf[:M], (rows.float() * torch.tensor(0.3, device="cuda")).to(torch.bfloat16))
    assert ws.last_launch()["kernel"] == "embed_kernel" and ws.device_status()["code"] == 0


def gradient64(ids, dy, V, scale, base=None):
    """The sums and their bound: n rows in fp32 are off by at most (n - 1) U sum|dy|, a product and a rounding follow."""
    inside = (ids >= 0) & (ids < V)
    at, x = ids[inside].long(), dy[inside].double()
    s, mag = (torch.zeros((V, dy.shape[1]), dtype=torch.float64, device="cuda") for _ in range(2))
    s.index_add_(0, at, x)
    mag.index_add_(0, at, x.abs())
    n = torch.zeros(V, dtype=torch.float64, device="cuda").index_add_(0, at, torch.ones_like(at, dtype=torch.float64))
    s, tol = s * scale, (n[:, None] + 2) * U * mag * abs(scale)
    if base is not None:
        s = s + base.double()
        tol = tol + U * s.abs()
    return s, tol + BF16 * (s.abs() + tol) + 1e-38, n > 0


# one token; up to 512 tokens, in one launch; one more; runs of ids over chunk ends; 16384 tokens and one more than the sort takes at
# once, several of its runs; one to three passes of digits; narrow rows (chunks share a block), rows of several slabs
@pytest.mark.parametrize("kind", ["text", "uniform", "one", "runs"])
@pytest.mark.parametrize("R,M,N,V", [(1, 1, 8, 1), (2, 7, 72, 3), (3, 300, 1032, 367), (1, 512, 520, 90), (2, 511, 40, 3000000),
                                     (1, 513, 4104, 77), (8, 1000, 64, 50), (4, 1025, 2056, 700),
                                     (2, 5000, 136, 40000), (1, 16384, 264, 65536), (5, 16385, 64, 8192), (2, 40000, 128, 600000),
                                     (8, 3000, 4096, 100), (1, 70000, 8, 5), (1, 33000, 40, 1100000)])
def test_gradient(ws, R, M, N, V, kind):
    r, g = rand(R + M + N + V)
    ids, dy = tokens(kind, M, R * V, g), r(M, N)
    buf = torch.full((R, V + 1, N), 3.0, dtype=torch.bfloat16, device="cuda")
    d = [b[:V] for b in buf]
    are.embedding_ar_backward(ids, dy, d, ws, scale=1.7)
    assert ws.device_status()["code"] == 0
    assert ws.last_launch()["kernel"] == ("embed_few_kernel" if M <= 512 else "embed_sort_kernel")
    scale = torch.tensor(1.7).item()
    want, tol, there = gradient64(ids, dy, R * V, scale)
    check(torch.cat(d), want, tol, "dtable")
    assert (torch.cat(d)[~there] == 0).all() and (buf[:, V] == 3).all()
    first = [t.clone() for t in d]
    are.embedding_ar_backward(ids.int(), dy, d, ws, scale=1.7)   # the same bits again, and from 32-bit ids
    assert all(torch.equal(a, b) for a, b in zip(first, d))
    # accumulating: touched rows grow, the others keep their bits
    base = [r(V, N) for _ in range(R)]
    d = [t.clone() for t in base]
    are.embedding_ar_backward(ids, dy, d, ws, scale=1.7, accumulate=True)
    want, tol, there = gradient64(ids, dy, R * V, scale, torch.cat(base))
    check(torch.cat(d), want, tol, "dtable, accumulated")
    assert torch.equal(torch.cat(d)[~there], torch.cat(base)[~there])


def test_gradient_against_differences(ws):
    """sum(dy * out) is linear in the table: a difference of 64-bit sums is the gradient itself."""
    r, g = rand(3)
    ids, dy = tokens("text", 50, 40, g), r(50, 16)
    d = [torch.empty((20, 16), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    are.embedding_ar_backward(ids, dy, d, ws, scale=0.5)
    _, tol, _ = gradient64(ids, dy, 40, 0.5)
    inside = (ids >= 0) & (ids < 40)

    def total(t):
        return (dy.double() * 0.5 * torch.where(inside[:, None], t[ids.clamp(0, 39)], 0.0)).sum()
    t, num = torch.zeros((40, 16), dtype=torch.float64, device="cuda"), torch.zeros((40, 16), dtype=torch.float64, device="cuda")
    for v in range(40):
        for j in range(16):
            t[v, j] = 1.0
            num[v, j] = total(t)
            t[v, j] = 0.0
    check(torch.cat(d), num, tol + 1e-12, "dtable by differences")


def test_values_that_are_not_finite(ws):
    """A NaN row reaches its own id's gradient and no other; rows without an id may hold anything."""
    r, g = rand(4)
    ids = torch.tensor([3, 1, -1, 3, 7, 1], device="cuda")
    dy = r(6, 64)
    dy[3, 5], dy[2] = float("nan"), float("inf")
    d = torch.empty((8, 64), dtype=torch.bfloat16, device="cuda")
    are.embedding_ar_backward(ids, dy, [d], ws)
    want, tol, _ = gradient64(ids[[1, 4, 5]], dy[[1, 4, 5]], 8, 1.0)
    assert d[3, 5].isnan() and d[3].isnan().sum() == 1
    keep = [0, 1, 2, 4, 5, 6, 7]
    check(d[keep], want[keep], tol[keep], "dtable")


def test_no_tokens_and_streams(ws):
    r, g = rand(5)
    empty, ids = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.empty(0, dtype=torch.int64, device="cuda")
    d = [torch.full((9, 64), 2.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    are.embedding_ar(ids, d, empty, ws)
    are.embedding_ar_backward(ids, empty, d, ws, accumulate=True)
    assert all((t == 2).all() for t in d)
    are.embedding_ar_backward(ids, empty, d, ws)
    assert all((t == 0).all() for t in d)
    # no token has an id
    are.embedding_ar_backward(torch.full((20,), -1, device="cuda"), r(20, 64), d, ws)
    assert all((t == 0).all() for t in d)
    s = torch.cuda.Stream()
    ids, dy = tokens("text", 200, 18, g), r(200, 64)
    s.wait_stream(torch.cuda.current_stream())
    are.embedding_ar_backward(ids, dy, d, ws, stream=s)
    torch.cuda.synchronize()
    want, tol, _ = gradient64(ids, dy, 18, 1.0)
    check(torch.cat(d), want, tol, "dtable")


def test_graph_replays(ws):
    r, g = rand(6)
    R, M, N, V = 2, 700, 256, 300
    tables, dy, ids = [r(V, N) for _ in range(R)], r(M, N), tokens("text", M, R * V, g)
    out, d = torch.empty_like(dy), [torch.empty((V, N), dtype=torch.bfloat16, device="cuda") for _ in range(R)]

    def call():
        are.embedding_ar(ids, tables, out, ws, scale=2.0)
        are.embedding_ar_backward(ids, dy, d, ws, scale=2.0)
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for k in range(3):
        r, g = rand(60 + k)
        ids.copy_(tokens("text", M, R * V, g))
        dy.copy_(r(M, N))
        graph.replay()
        torch.cuda.synchronize()
        want, tol, _ = gradient64(ids, dy, R * V, 2.0)
        check(torch.cat(d), want, tol, "dtable")
        inside = (ids >= 0) & (ids < R * V)
        assert torch.equal(out, torch.where(inside[:, None], torch.cat(tables)[ids.clamp(0, R * V - 1)] * 2, 0.0).to(torch.bfloat16))


def test_offsets_past_32_bits():
    """A table of more than 2^32 bytes, and more than 2^32 bytes of dy."""
    need_gpu()
    N, V, M = 8200, (1 << 18) + 7, (1 << 18) + 3
    r, g = rand(7)
    big = torch.zeros((V, N), dtype=torch.bfloat16, device="cuda")
    big[V - 1] = r(1, N)[0]
    ids = torch.full((M,), -1, device="cuda")
    ids[0], ids[M - 1], ids[M - 2] = V - 1, V - 1, 3
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    with are.Workspace(R_max=1, M_max=M, N_max=8200) as ws:
        are.embedding_ar(ids, [big], out, ws)
        assert torch.equal(out[0], big[V - 1]) and torch.equal(out[M - 1], big[V - 1]) and (out[1:M - 1] == 0).all()
        dy = torch.zeros_like(out)
        dy[[0, M - 2, M - 1]] = r(3, N)
        are.embedding_ar_backward(ids, dy, [big], ws)
        assert ws.device_status()["code"] == 0
    assert torch.equal(big[3], dy[M - 2])
    assert torch.equal(big[V - 1], (dy[0].float() + dy[M - 1].float()).to(torch.bfloat16))
    assert (big[4:V - 1] == 0).all() and (big[:3] == 0).all()


@pytest.mark.parametrize("N", [8, 64, 2056, 16384, 32768])
def test_workspaces_no_wider_than_the_row(N):
    """Partial rows of every chunk fit a workspace made for this width."""
    need_gpu()
    r, g = rand(8)
    M = 9000 if N < 10000 else 3000
    ids, dy = tokens("runs", M, 100, g), r(M, N)
    d = torch.empty((100, N), dtype=torch.bfloat16, device="cuda")
    with are.Workspace(R_max=1, M_max=M, N_max=N) as w:
        are.embedding_ar_backward(ids, dy, [d], w)
        assert w.device_status()["code"] == 0
    want, tol, _ = gradient64(ids, dy, 100, 1.0)
    check(d, want, tol, "dtable")


def test_refusals(ws):
    r, g = rand(9)
    ids, dy, d = torch.zeros(6, dtype=torch.int64, device="cuda"), r(6, 64), [r(5, 64), r(5, 64)]
    out = torch.empty_like(dy)
    for kw in (dict(ids=ids[:5]), dict(ids=ids.float()), dict(ids=ids.cpu()), dict(d=[d[0], d[1][:3]]), dict(d=[]),
               dict(dy=dy[:, :32]), dict(dy=dy.float()), dict(d=[t.float() for t in d])):
        a = dict(ids=ids, dy=dy, d=d)
        a.update(kw)
        with pytest.raises(ValueError):
            are.embedding_ar(a["ids"], a["d"], a["dy"], ws)
        with pytest.raises(ValueError):
            are.embedding_ar_backward(a["ids"], a["dy"], a["d"], ws)
    for scale in (float("nan"), float("inf")):
        with pytest.raises(are.AreError):
            are.embedding_ar(ids, d, out, ws, scale=scale)
        with pytest.raises(are.AreError):
            are.embedding_ar_backward(ids, dy, d, ws, scale=scale)
    both = r(11, 64)
    for tables, grad in (([d[0], d[0]], dy), ([both[:5], both[4:9]], dy), ([both[:5], both[5:10]], both[4:10])):   # overlapping
        with pytest.raises(are.AreError) as e:
            are.embedding_ar_backward(ids, grad, tables, ws)
        assert e.value.status == are.EINVAL
    with pytest.raises(are.AreError):
        are.embedding_ar(ids, [both[:5], both[5:10]], both[4:10], ws)
    odd = torch.empty((6, 60), dtype=torch.bfloat16, device="cuda")
    with pytest.raises(are.AreError):
        are.embedding_ar(ids, [odd], torch.empty_like(odd), ws)
    for caps in (dict(R_max=1), dict(M_max=5), dict(N_max=32)):
        c = dict(R_max=2, M_max=6, N_max=64)
        c.update(caps)
        with are.Workspace(**c) as other:
            with pytest.raises(are.AreError) as e:
                are.embedding_ar_backward(ids, dy, d, other)
            assert e.value.status == are.ECAPACITY


# one CTA's most tokens and a cluster's first; a part with no token; four items a thread and more; all that a cluster sorts at once, one
# more, several runs; one to three passes
@pytest.mark.parametrize("kind", ["text", "uniform", "one", "runs"])
@pytest.mark.parametrize("R,M,N,V", [(2, 2048, 64, 900), (2, 2049, 64, 900), (1, 7169, 40, 1), (3, 32768, 64, 5000), (1, 32769, 64, 70000),
                                     (4, 131072, 16, 300), (1, 131073, 8, 1100000), (2, 300000, 8, 9000)])
def test_gradient_by_a_cluster_s_sort(R, M, N, V, kind):
    need_gpu()
    with are.Workspace(R_max=R, M_max=M, N_max=N) as ws:
        test_gradient(ws, R, M, N, V, kind)


def test_gradients_back_to_back(ws):
    """Calls in a row, whose kernels overlap at their ends, on tables that the call before wrote and read: zeros of the next
    call come after the sums of this one."""
    r, g = rand(11)
    M, N, V = 6000, 1032, 3000
    d = [torch.empty(V, N, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    calls = []
    for k in range(6):
        ids, dy = tokens("text" if k % 2 else "uniform", M, 2 * V, g), r(M, N)
        calls.append((ids, dy, torch.zeros(M, N, dtype=torch.bfloat16, device="cuda")))
    torch.cuda.synchronize()
    for ids, dy, out in calls:
        are.embedding_ar_backward(ids, dy, d, ws)
        are.embedding_ar(ids, d, out, ws)
    torch.cuda.synchronize()
    for ids, dy, out in calls:
        want, tol, _ = gradient64(ids, dy, 2 * V, 1.0)
        here = (ids >= 0) & (ids < 2 * V)
        at = ids.clamp(0, 2 * V - 1)
        check(out, want[at] * here[:, None], torch.where(here[:, None], tol[at], 1e-38), "rows read back")


def test_gradient_of_a_vocabulary_past_30_bits():
    """Four passes of digits in several runs: a pass reads what other CTAs wrote where the pass before the last had read."""
    need_gpu()
    R, V, M, N = 8, 140_000_000, 140_000, 8
    r, g = rand(17)
    ids = torch.randint(0, R * V, (M,), generator=g, device="cuda")
    ids[::7] = ids[3]
    dy = r(M, N)
    d = [torch.full((V, N), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(R)]
    with are.Workspace(R_max=R, M_max=M, N_max=N) as ws:
        are.embedding_ar_backward(ids, dy, d, ws)
        assert ws.device_status()["code"] == 0
    there, at = torch.unique(ids, return_inverse=True)
    want, tol, _ = gradient64(at, dy, len(there), 1.0)
    got = torch.stack([t[(there - k * V).clamp(0, V - 1)] for k, t in enumerate(d)])
    rank = torch.div(there, V, rounding_mode="floor")
    check(got[rank, torch.arange(len(there), device="cuda")], want, tol, "dtable")
    for k, t in enumerate(d):   # and nothing else
        rows = t.view(torch.int64).view(V, 2)
        assert int((rows != 0).any(1).sum()) <= int((rank == k).sum())
