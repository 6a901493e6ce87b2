"""The embedding, LayerNorm and the cross entropy as a training step and a scoring call use them."""
import os
import subprocess
import sys
import textwrap

import pytest
import torch

import all_reduce_epilogue_gb300 as are
from tests import ends_ref as ref
from tests.gpu_util import need_gpu
from tests.test_gpu_embedding import gradient64

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


class Step:
    """Embedding, a layer's all-reduce with LayerNorm, the output layer and its loss, and back, with the table tied to the
    output layer: the embedding's gradient is added to dw."""

    def __init__(self, R, M, K, N, seed, stream=None):
        self.stream = stream
        self.ws = are.Workspace(R_max=R, M_max=M, N_max=K, K_max=K, vocab_piece=256)
        bf = dict(dtype=torch.bfloat16, device="cuda")
        self.shape, self.V = (R, M, K, N), R * N - 3
        self.ids, self.targets = (torch.zeros(M, dtype=torch.int64, device="cuda") for _ in range(2))
        self.table = torch.empty((R, N, K), **bf)
        self.parts = [torch.empty((M, K), **bf) for _ in range(R)]   # what the layer between leaves on the ranks
        self.gamma, self.beta, self.dloss = torch.empty(K, device="cuda"), torch.empty(K, device="cuda"), torch.empty(M, device="cuda")
        self.x, self.h, self.y, self.dy, self.dx = (torch.empty((M, K), **bf) for _ in range(5))
        self.loss, self.lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
        self.dw, self.dgamma, self.dbeta = torch.empty((R, N, K), **bf), torch.empty(K, device="cuda"), torch.empty(K, device="cuda")
        self.fill(seed)

    def fill(self, seed):
        R, M, K, N = self.shape
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
        self.ids.copy_(torch.randint(0, self.V, (M,), generator=g, device="cuda") // 2)
        self.targets.copy_(torch.randint(0, self.V, (M,), generator=g, device="cuda"))
        self.ids[-2:], self.targets[-2:] = -1, -100    # padding
        self.table.copy_(r(R, N, K) * 0.1)
        for p in self.parts:
            p.copy_(r(M, K) * 0.1)
        self.gamma.copy_(1 + 0.1 * r(K))
        self.beta.copy_(0.1 * r(K))
        self.dloss.copy_(torch.full((M,), 1.0 / (M - 2), device="cuda"))
        self.dx.copy_(self.x)

    def forward(self):
        w, s = list(self.table), self.stream
        are.embedding_ar(self.ids, w, self.x, self.ws, scale=8.0, stream=s)
        are.allreduce_layernorm(self.parts, self.x, self.gamma, self.beta, ref.EPS, self.y, self.ws, residual_out=self.h, stream=s)
        are.gemm_cross_entropy(self.y, w, self.targets, self.loss, self.lse, self.ws, vocab=self.V, stream=s)

    def backward(self):
        w, dw, s = list(self.table), list(self.dw), self.stream
        are.gemm_cross_entropy_backward(self.y, w, self.targets, self.lse, self.dloss, self.dy, dw, self.ws, vocab=self.V, stream=s)
        are.allreduce_layernorm_backward([self.dy], self.h, self.gamma, ref.EPS, self.dx, self.dgamma, self.dbeta, self.ws, stream=s)
        are.embedding_ar_backward(self.ids, self.dx, dw, self.ws, scale=8.0, accumulate=True, stream=s)

    def run(self):
        self.forward()
        self.backward()

    def results(self):
        return [t.clone() for t in (self.x, self.h, self.y, self.loss, self.lse, self.dy, self.dx, self.dgamma, self.dbeta, self.dw)]

    def check(self):
        """Every stage against 64 bits of what it was given."""
        R, M, K, N = self.shape
        assert self.ws.device_status()["code"] == 0
        full = self.table.flatten(0, 1)
        inside = self.ids >= 0
        assert torch.equal(self.x, torch.where(inside[:, None], full[self.ids.clamp(min=0)] * 8, 0.0).to(torch.bfloat16))
        y, tol, h, tol_h = ref.layernorm64(self.parts, self.x, self.gamma, self.beta)
        ref.check(self.h, h, tol_h, "h")
        ref.check(self.y, y, tol, "y")
        (loss, tl), (lse, ts), (dy, td), (dw, tw) = ref.cross_entropy64(self.y, list(self.table), self.targets, self.V, self.dloss)
        ref.check(self.loss, loss, tl, "loss")
        ref.check(self.lse, lse, ts, "lse")
        ref.check(self.dy, dy, td, "dy")
        want = ref.layernorm_backward64([self.dy], self.h, self.gamma, None)
        for got, v, t, what in zip((self.dx, self.dgamma, self.dbeta), want[::2], want[1::2], ("dx", "dgamma", "dbeta")):
            ref.check(got, v, t, what)
        s, t, there = gradient64(self.ids, self.dx, R * N, 8.0)
        # dw was rounded to bf16 (its bound) before the embedding's gradient was added, and where it was, once more
        want, tol = dw.flatten(0, 1) + s, tw.flatten(0, 1) + t
        tol = tol + torch.where(there[:, None], ref.BF16 * (want.abs() + tol), 0.0)
        ref.check(self.dw.flatten(0, 1), want, tol, "dw")


@pytest.mark.parametrize("R,M,K,N", [(2, 20, 64, 60), (4, 300, 264, 333), (8, 1000, 512, 300), (1, 130, 4096, 700)])
def test_training_step(R, M, K, N):
    need_gpu()
    s = Step(R, M, K, N, 1)
    with s.ws:
        s.run()
        s.check()
        # captured and replayed with other inputs
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            s.run()
        for k in range(3):
            s.fill(2 + k)
            graph.replay()
            torch.cuda.synchronize()
            s.check()


def test_two_graphs_on_one_workspace():
    """Two captured steps that use the same workspace, replayed in turn on a stream: the bits of either alone."""
    need_gpu()
    a, b = Step(2, 70, 128, 200, 1), Step(2, 50, 128, 150, 2)
    b.ws.close()
    b.ws = a.ws
    with a.ws:
        want = []
        for s in (a, b):
            s.run()
            want.append(s.results())
        graphs = []
        for s in (a, b):
            graphs.append(torch.cuda.CUDAGraph())
            with torch.cuda.graph(graphs[-1]):
                s.run()
        for k in (0, 1, 1, 0, 0, 1):
            graphs[k].replay()
        torch.cuda.synchronize()
        for s, w in zip((a, b), want):
            for x, y in zip(s.results(), w):
                assert torch.equal(x, y)


def test_two_streams_with_a_workspace_each():
    """The same steps at once on two streams, each with its own workspace and tensors: the bits of either alone."""
    need_gpu()
    steps = [Step(4, 300, 512, 400, 1, torch.cuda.Stream()), Step(2, 200, 1024, 900, 2, torch.cuda.Stream())]
    torch.cuda.synchronize()
    want = []
    for s in steps:
        s.run()
        torch.cuda.synchronize()
        want.append(s.results())
    torch.cuda.synchronize()
    for _ in range(20):
        for s in steps:
            s.run()
    torch.cuda.synchronize()
    for s, w in zip(steps, want):
        assert s.ws.device_status()["code"] == 0
        for x, y in zip(s.results(), w):
            assert torch.equal(x, y)
        s.ws.close()


def test_scoring_beside_other_operations():
    """The loss on a workspace between the framework's own GEMM and norm calls on it: all keep their bits."""
    need_gpu()
    R, M, K, N = 2, 64, 256, 300
    g = torch.Generator(device="cuda").manual_seed(3)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    A, B = [r(M, K) for _ in range(R)], [r(K, K) * 0.05 for _ in range(R)]
    w, gamma, t = [r(N, K) for _ in range(R)], torch.ones(K, device="cuda"), torch.arange(M, device="cuda")
    out, y = torch.empty((M, K), dtype=torch.bfloat16, device="cuda"), torch.empty((M, K), dtype=torch.bfloat16, device="cuda")
    loss, lse = torch.empty(M, device="cuda"), torch.empty(M, device="cuda")
    with are.Workspace(R_max=R, M_max=M, N_max=K, K_max=K, vocab_piece=256) as ws:
        def run():
            are.gemm_ar(A, B, out, ws)
            are.allreduce_rmsnorm([out], None, gamma, 1e-6, y, ws)
            are.gemm_cross_entropy(y, w, t, loss, lse, ws)
        run()
        first = [x.clone() for x in (out, y, loss, lse)]
        ref.check(loss, *ref.cross_entropy64(y, w, t, R * N)[0], "loss")
        for _ in range(5):
            run()
        for a, b in zip(first, (out, y, loss, lse)):
            assert torch.equal(a, b)
        assert ws.device_status()["code"] == 0


def test_first_calls_captured():
    """In a fresh process, the first call of each operation on a workspace is made inside a capture."""
    need_gpu()
    code = textwrap.dedent("""
        import sys
        import torch
        sys.path.insert(0, ROOT)
        import all_reduce_epilogue_gb300 as are
        bf = dict(dtype=torch.bfloat16, device="cuda")
        x, h, dh, y = (torch.full((20, 256), 2.0, **bf) for _ in range(4))
        w, dw, d = torch.zeros((64, 256), **bf), torch.ones((64, 256), **bf), torch.ones((64, 256), **bf)
        one, dg, db = torch.ones(256, device="cuda"), torch.zeros(256, device="cuda"), torch.zeros(256, device="cuda")
        ids, loss, lse = torch.arange(20, device="cuda"), torch.zeros(20, device="cuda"), torch.zeros(20, device="cuda")
        g = torch.ones(20, device="cuda")
        spaces = [are.Workspace(1, 20, 256, K_max=256, vocab_piece=256) for _ in range(6)]
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            are.allreduce_layernorm([x], None, one, one, 1e-5, y, spaces[0])
            are.allreduce_layernorm_backward([x], h, one, 1e-5, dh, dg, db, spaces[1])
            are.gemm_cross_entropy(x, [w], ids, loss, lse, spaces[2])
            are.gemm_cross_entropy_backward(x, [w], ids, lse, g, h, [dw], spaces[3])
            are.embedding_ar_backward(ids, x, [d], spaces[4])
            are.embedding_ar(ids, [d], x, spaces[5], scale=2.0)
        graph.replay()
        torch.cuda.synchronize()
        for ws in spaces:
            assert ws.device_status()["code"] == 0
        log64 = torch.log(torch.tensor(64.0)).item()
        assert bool((y == 1).all()) and bool((db == 40).all()) and bool((dg == 0).all())
        assert bool(((loss - log64).abs() < 1e-5).all()) and bool((h == 0).all())
        want = torch.full((64,), 40 / 64, device="cuda")
        want[:20] -= 2
        assert bool(((dw.float() - want[:, None]).abs() <= 2.0 ** -7 * want[:, None].abs()).all())
        assert bool((d[:20] == 2).all()) and bool((d[20:] == 0).all()) and bool((x == 4).all())
        print("ok")
    """).replace("ROOT", repr(ROOT))
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "ok" in r.stdout, r.stdout + r.stderr


def test_workspaces_without_what_one_operation_needs():
    """The partial rows of LayerNorm's gradients and the sorted tokens take no memory before a call needs them."""
    need_gpu()

    def held():
        torch.cuda.synchronize()
        return torch.cuda.mem_get_info()[0]
    bf = dict(dtype=torch.bfloat16, device="cuda")
    M, N = 1 << 20, 16384
    x, dh, g = torch.randn((600, 64), device="cuda").to(torch.bfloat16), torch.empty((600, 64), **bf), torch.ones(64, device="cuda")
    dg, db, ids = torch.empty_like(g), torch.empty_like(g), torch.arange(600, device="cuda") % 50
    table = torch.empty((50, 64), **bf)
    with are.Workspace(R_max=1, M_max=600, N_max=64) as ws:   # (kernels are loaded by their first launch)
        for rows in (64, 600):
            are.allreduce_layernorm_backward([x[:rows]], x[:rows], g, 1e-5, dh[:rows], dg, db, ws)
        for rows in (512, 600):
            are.embedding_ar_backward(ids[:rows], x[:rows], [table], ws)
    before = held()
    with are.Workspace(R_max=1, M_max=64, N_max=N) as ws:
        made = held()
        assert before - made < 30 << 20   # 20 MB for the RMSNorm's partial sums, 4 MB of staging, 2 MB of tokens
        are.allreduce_layernorm_backward([x[:64]], x[:64], g, 1e-5, dh[:64], None, None, ws)
        assert held() == made
        are.allreduce_layernorm_backward([x[:64]], x[:64], g, 1e-5, dh[:64], dg, db, ws)
        assert 38 << 20 <= made - held() < 50 << 20   # 4 * 16384 * 152 words are 38 MiB
    before = held()
    with are.Workspace(R_max=1, M_max=M, N_max=64) as ws:
        made = held()
        assert before - made < 270 << 20  # 256 MB of staging
        are.embedding_ar_backward(ids[:512], x[:512], [table], ws)
        assert held() == made
        are.embedding_ar_backward(ids, x, [table], ws)
        assert made - held() > 17 * M
        now = held()
        are.embedding_ar_backward(ids, x, [table], ws)
        are.allreduce_layernorm_backward([x], x, g, 1e-5, dh, dg, db, ws)
        assert held() == now
        want = torch.zeros((50, 64), dtype=torch.float64, device="cuda").index_add_(0, ids, x.double())
        assert ((table.double() - want).abs() <= want.abs() * 2.0 ** -8 + 1e-4).all()


def test_capacities_past_64_bits_are_refused():
    need_gpu()
    for M, N, K in ((1 << 60, 8, 0), (1 << 62, 32768, 0), (1 << 61, 8, 8), (8, 1 << 62, 8)):
        with pytest.raises(are.AreError) as e:
            are.Workspace(R_max=8, M_max=M, N_max=N, K_max=K)
        assert e.value.status == are.ENOMEM


def test_a_refused_allocation_leaves_no_error_behind():
    """A workspace, or the cross entropy's buffers, that the device has no room for: a status, and nothing that the next
    launch of the process reports."""
    need_gpu()
    x = torch.ones(8, device="cuda")
    with are.Workspace(R_max=1, M_max=65536, N_max=8, K_max=8) as ws:
        with pytest.raises(are.AreError) as e:
            ws.set_vocab_piece(1 << 27)      # 2^45 bytes
        assert e.value.status == are.ENOMEM
        assert (x + 1 == 2).all()
        with pytest.raises(are.AreError) as e:
            are.Workspace(R_max=1, M_max=1 << 40, N_max=8)
        assert e.value.status == are.ENOMEM
        assert (x * 2 == 2).all()
        ws.set_vocab_piece(256)
        h = torch.zeros((4, 8), dtype=torch.bfloat16, device="cuda")
        loss, lse, t = torch.empty(4, device="cuda"), torch.empty(4, device="cuda"), torch.zeros(4, dtype=torch.int64, device="cuda")
        are.gemm_cross_entropy(h, [h], t, loss, lse, ws)
        assert ((loss - torch.log(torch.tensor(4.0, device="cuda"))).abs() < 1e-6).all()
