"""Cases of the operators at both ends of a tensor-parallel model and of its LayerNorm.

Six operators:

* ``layernorm``: all-reduce of R bf16 partials, residual add and LayerNorm;
* ``layernorm_backward``: its backward pass, whose output gradient arrives as R
  bf16 partials;
* ``embedding``: lookup in a table whose vocabulary is split over R ranks, scaled;
* ``embedding_backward``: the gradient of every rank's part of the table;
* ``loss``: softmax cross entropy of an output layer whose vocabulary is split
  over R ranks, the logits not kept;
* ``loss_step``: the same with the gradients of the hidden states and of every
  rank's weights.

``run`` computes them with elementary torch operations in 32 bits, or, where
``own`` is true, with the calls of ``all_reduce_epilogue_gb300``.
"""
import math

import torch

own = False
EPS = 1e-5

_workspaces = {}


def listed():
    return [
        # the norm after a row-parallel linear, one token, 8 ranks: the smallest decode call
        {"name": "layernorm token R8", "op": "layernorm", "R": 8, "M": 1, "N": 7168, "residual": True,
         "residual_out": True, "beta": True},
        # a prompt of 4096 tokens, 8 ranks
        {"name": "layernorm prompt R8", "op": "layernorm", "R": 8, "M": 4096, "N": 7168, "residual": True,
         "residual_out": True, "beta": True},
        # odd row count, width no multiple of a tile, the last layer (no residual gradient), a norm without bias
        {"name": "layernorm backward odd R3", "op": "layernorm_backward", "R": 3, "M": 1001, "N": 5000, "dres": False,
         "beta": False},
        # a training step's full batch on one rank
        {"name": "layernorm backward batch R1", "op": "layernorm_backward", "R": 1, "M": 16384, "N": 4096, "dres": True,
         "beta": True},
        # the embedding of a few tokens of a decode batch
        {"name": "embedding tokens R2", "op": "embedding", "R": 2, "M": 5, "N": 2048, "Vs": 16000, "scale": 1.0,
         "wide": False},
        # the embedding of a training batch, scaled by sqrt(N) as tied tables are
        {"name": "embedding batch R8", "op": "embedding", "R": 8, "M": 16384, "N": 4096, "Vs": 8192, "scale": 64.0,
         "wide": True},
        # a short fine-tuning step: ragged rows, an odd vocabulary
        {"name": "embedding backward short R3", "op": "embedding_backward", "R": 3, "M": 300, "N": 1032, "Vs": 3667,
         "scale": 1.0, "wide": False},
        # a training batch's gradient: a few tokens make up much of the text
        {"name": "embedding backward batch R8", "op": "embedding_backward", "R": 8, "M": 16384, "N": 4096, "Vs": 8192,
         "scale": 64.0, "wide": True},
        # scoring one token: the weights are read once
        {"name": "loss token R2", "op": "loss", "R": 2, "M": 1, "K": 2048, "Vs": 16000, "vocab": 32000, "wide": False},
        # evaluation of a batch
        {"name": "loss batch R8", "op": "loss", "R": 8, "M": 4096, "K": 4096, "Vs": 8192, "vocab": 65536, "wide": True},
        # a short fine-tuning step on an odd vocabulary, padded to whole ranks
        {"name": "loss step ragged R3", "op": "loss_step", "R": 3, "M": 77, "K": 1000, "Vs": 3667, "vocab": 11000,
         "wide": False},
        # a training step's output layer and loss
        {"name": "loss step batch R8", "op": "loss_step", "R": 8, "M": 4096, "K": 4096, "Vs": 8192, "vocab": 65536,
         "wide": True},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], spread over the logarithm."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + step))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(["layernorm", "layernorm_backward", "embedding", "embedding_backward", "loss", "loss_step"])
    R = rng.randint(1, 8)
    if op == "layernorm":
        N = _log(rng, 64, 16384, 8)
        M = _log(rng, 1, min(16384, max(1, 8 * 4096 * 7168 // (R * N))))
        return {"op": op, "R": R, "M": M, "N": N, "residual": rng.random() < 0.8, "residual_out": rng.random() < 0.8,
                "beta": rng.random() < 0.8}
    if op == "layernorm_backward":
        N = _log(rng, 64, 16384, 8)
        M = _log(rng, 1, min(16384, max(1, 3 * 16384 * 4096 // ((R + 2) * N))))
        return {"op": op, "R": R, "M": M, "N": N, "dres": rng.random() < 0.7, "beta": rng.random() < 0.8}
    if op.startswith("embedding"):
        N = _log(rng, 64, 8192, 8)
        M = _log(rng, 1, min(16384, 16384 * 4096 // N))
        Vs = _log(rng, 100, max(100, min(131072, 65536 * 4096 // N) // R))
        return {"op": op, "R": R, "M": M, "N": N, "Vs": Vs, "scale": rng.choice([1.0, math.sqrt(N)]),
                "wide": rng.random() < 0.5}
    K = _log(rng, 64, 8192, 8)
    Vs = _log(rng, 100, 65536 // R)
    M = _log(rng, 1, max(1, min(4096, 4096 * 65536 * 4096 // (R * Vs * K))))
    return {"op": op, "R": R, "M": M, "K": K, "Vs": Vs, "vocab": R * Vs - rng.choice([0, rng.randrange(Vs)]),
            "wide": rng.random() < 0.5}


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    R, M, op = case["R"], case["M"], case["op"]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale)

    def channels(n):
        """Per-channel magnitudes: most near one, a few outlier channels."""
        c = torch.exp(normal(n, scale=0.4))
        return torch.where(torch.rand(n, generator=gen, device="cuda") < 0.004, c * 20, c)

    def text(vocab, missing):
        """M tokens: few make up most of them, those spread over the vocabulary; some positions hold none."""
        u = torch.rand(M, generator=gen, device="cuda", dtype=torch.float64)
        rank = torch.exp(u * math.log(vocab + 1)).long() - 1  # probability about 1 / (rank log vocab)
        ids = (rank.clamp(0, vocab - 1) * 7919 + 13) % vocab
        if M > 8:
            ids[-(M // 16 + 1):] = missing
        return ids if case["wide"] else ids.int()

    def bf16(*shape):
        return torch.empty(shape, dtype=torch.bfloat16, device="cuda")

    s = dict(case)
    if op == "layernorm":
        N = case["N"]
        x, ch = bf16(R, M, N), channels(N)
        for r in range(R):
            x[r] = normal(M, N) * ch + 0.3
        res = (normal(M, N) * ch * 2 + normal(M, 1)).to(torch.bfloat16) if case["residual"] else None
        if M > 8:  # rows that pad a batch
            x[:, -2:] = 0
            if res is not None:
                res[-2:] = 0
        s.update(x=x, partials=list(x), res=res, gamma=1 + normal(N, scale=0.1), out=bf16(M, N),
                 bias=normal(N, scale=0.1) if case["beta"] else None,
                 res_out=bf16(M, N) if case["residual_out"] else None)
    elif op == "layernorm_backward":
        N = case["N"]
        dy = bf16(R, M, N)
        for r in range(R):
            dy[r] = normal(M, N, scale=1e-2)
        if M > 8:  # rows that take no part in the loss
            dy[:, M // 2] = 0
        s.update(dy=dy, partials=list(dy), h=(normal(M, N) * channels(N) * 3 + normal(M, 1)).to(torch.bfloat16),
                 gamma=1 + normal(N, scale=0.1), dh=bf16(M, N),
                 d_res=normal(M, N, scale=1e-2).to(torch.bfloat16) if case["dres"] else None,
                 dgamma=torch.empty(N, dtype=torch.float32, device="cuda"),
                 dbeta=torch.empty(N, dtype=torch.float32, device="cuda") if case["beta"] else None)
    elif op.startswith("embedding"):
        N, Vs = case["N"], case["Vs"]
        s.update(ids=text(R * Vs, -1))
        if op == "embedding":
            table = bf16(R, Vs, N)
            for r in range(R):
                table[r] = normal(Vs, N, scale=0.02)
            s.update(table=table, tables=list(table), out=bf16(M, N))
        else:
            dtable = bf16(R, Vs, N)
            s.update(dy=normal(M, N, scale=1e-2).to(torch.bfloat16), dtable=dtable, dtables=list(dtable))
    else:
        K, Vs, vocab = case["K"], case["Vs"], case["vocab"]
        w = bf16(R, Vs, K)
        for r in range(R):
            w[r] = normal(Vs, K, scale=1.5 / math.sqrt(K))
        targets = text(vocab, -100)
        # what a trained model gives: half of the tokens are foreseen, more or less surely
        sure = 6 * torch.rand(M, generator=gen, device="cuda") * (torch.rand(M, generator=gen, device="cuda") < 0.5)
        h = normal(M, K) + sure[:, None] * w.view(R * Vs, K)[targets.clamp(min=0).long()].float()
        weight = (targets >= 0).float() * (0.5 + torch.rand(M, generator=gen, device="cuda"))
        s.update(w=w, weights=list(w), targets=targets, h=h.to(torch.bfloat16),
                 dloss=weight / (targets >= 0).sum().clamp(min=1), dh=bf16(M, K), dw=bf16(R, Vs, K),
                 loss=torch.empty(M, dtype=torch.float32, device="cuda"),
                 lse=torch.empty(M, dtype=torch.float32, device="cuda"))
        s["dweights"] = list(s["dw"])
    if own:
        s["ws"] = _workspace("loss" if op.startswith("loss") else "rows")
    return s


def _workspace(kind):
    """One workspace of each kind for the program."""
    import all_reduce_epilogue_gb300 as are
    if kind not in _workspaces:
        _workspaces[kind] = (are.Workspace(R_max=8, M_max=16384, N_max=16384) if kind == "rows" else
                             are.Workspace(R_max=8, M_max=4096, N_max=8, K_max=8192, vocab_piece=8192))
    return _workspaces[kind]


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "layernorm":
        h = s["x"].float().sum(0)
        if s["res"] is not None:
            h = h + s["res"].float()
        c = h - h.mean(-1, keepdim=True)
        y = c * torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS) * s["gamma"]
        if s["bias"] is not None:
            y = y + s["bias"]
        out = {"y": y.to(torch.bfloat16)}
        if s["residual_out"]:
            out["h"] = h.to(torch.bfloat16)
        return out
    if op == "layernorm_backward":
        dy, h = s["dy"].float().sum(0), s["h"].float()
        c = h - h.mean(-1, keepdim=True)
        inv = torch.rsqrt((c * c).mean(-1, keepdim=True) + EPS)
        xhat, g = c * inv, dy * s["gamma"]
        dh = inv * (g - g.mean(-1, keepdim=True) - xhat * (g * xhat).mean(-1, keepdim=True))
        if s["d_res"] is not None:
            dh = dh + s["d_res"].float()
        out = {"dh": dh.to(torch.bfloat16), "dgamma": (dy * xhat).sum(0)}
        if s["beta"]:
            out["dbeta"] = dy.sum(0)
        return out
    if op == "embedding":
        table = s["table"].flatten(0, 1)
        ok = (s["ids"] >= 0) & (s["ids"] < table.shape[0])
        rows = table[s["ids"].clamp(0, table.shape[0] - 1).long()].float() * s["scale"]
        return torch.where(ok[:, None], rows, torch.zeros_like(rows)).to(torch.bfloat16)
    if op == "embedding_backward":
        R, Vs, N = s["dtable"].shape
        ok = (s["ids"] >= 0) & (s["ids"] < R * Vs)
        d = torch.zeros((R * Vs, N), dtype=torch.float32, device="cuda")
        d.index_add_(0, s["ids"].clamp(0, R * Vs - 1).long(), s["dy"].float() * ok[:, None])
        return (d * s["scale"]).to(torch.bfloat16).view(R, Vs, N)
    h, w = s["h"].float(), s["w"].flatten(0, 1)[:s["vocab"]].float()
    logits = h @ w.T
    top = logits.amax(-1, keepdim=True)
    lse = (top + torch.log(torch.exp(logits - top).sum(-1, keepdim=True)))[:, 0]
    ok = (s["targets"] >= 0) & (s["targets"] < s["vocab"])
    at = s["targets"].clamp(0, s["vocab"] - 1).long()[:, None]
    out = {"loss": torch.where(ok, lse - logits.gather(1, at)[:, 0], torch.zeros_like(lse)), "lse": lse}
    if op == "loss_step":
        g = torch.where(ok, s["dloss"], torch.zeros_like(lse))[:, None]
        d = torch.exp(logits - lse[:, None]) * g
        d.scatter_add_(1, at, -g)
        dw = torch.zeros(s["w"].shape, dtype=torch.bfloat16, device="cuda")
        dw.flatten(0, 1)[:s["vocab"]] = d.T @ h
        out.update(dh=(d @ w).to(torch.bfloat16), dw=dw)
    return out


def _run_own(s):
    import all_reduce_epilogue_gb300 as are
    op = s["op"]
    if op == "layernorm":
        are.allreduce_layernorm(s["partials"], s["res"], s["gamma"], s["bias"], EPS, s["out"], s["ws"],
                                residual_out=s["res_out"])
        return {"y": s["out"], "h": s["res_out"]} if s["residual_out"] else {"y": s["out"]}
    if op == "layernorm_backward":
        are.allreduce_layernorm_backward(s["partials"], s["h"], s["gamma"], EPS, s["dh"], s["dgamma"], s["dbeta"], s["ws"],
                                         dres=s["d_res"])
        out = {"dh": s["dh"], "dgamma": s["dgamma"]}
        if s["beta"]:
            out["dbeta"] = s["dbeta"]
        return out
    if op == "embedding":
        are.embedding_ar(s["ids"], s["tables"], s["out"], s["ws"], scale=s["scale"])
        return s["out"]
    if op == "embedding_backward":
        are.embedding_ar_backward(s["ids"], s["dy"], s["dtables"], s["ws"], scale=s["scale"])
        return s["dtable"]
    are.gemm_cross_entropy(s["h"], s["weights"], s["targets"], s["loss"], s["lse"], s["ws"], vocab=s["vocab"])
    out = {"loss": s["loss"], "lse": s["lse"]}
    if op == "loss_step":
        are.gemm_cross_entropy_backward(s["h"], s["weights"], s["targets"], s["lse"], s["dloss"], s["dh"], s["dweights"],
                                        s["ws"], vocab=s["vocab"])
        out.update(dh=s["dh"], dw=s["dw"])
    return out


def work(case):
    R, M, op = case["R"], case["M"], case["op"]
    if op == "layernorm":
        N = case["N"]
        return {"bytes": M * N * 2 * (R + 1 + case["residual"] + case["residual_out"]) + 4 * N * (1 + case["beta"]),
                "flops": M * N * (R + 9)}
    if op == "layernorm_backward":
        N = case["N"]
        return {"bytes": M * N * 2 * (R + 2 + case["dres"]) + 4 * N * (2 + case["beta"]), "flops": M * N * (R + 16)}
    index = M * (8 if case["wide"] else 4)
    if op == "embedding":
        return {"bytes": M * case["N"] * 4 + index, "flops": M * case["N"]}
    if op == "embedding_backward":
        return {"bytes": M * case["N"] * 2 + R * case["Vs"] * case["N"] * 2 + index, "flops": 2 * M * case["N"]}
    K, V = case["K"], R * case["Vs"]
    once = (M * K + case["vocab"] * K) * 2 + index + M * 8
    if op == "loss":
        return {"bytes": once, "flops": 2 * M * case["vocab"] * K}
    # forward, and the gradients of both factors; the logits, which are not kept, a second time
    return {"bytes": once + (M * K + V * K) * 2 + M * 4, "flops": 8 * M * case["vocab"] * K}


def exact(case, seed):
    """The operators from their definitions in 64 bits."""
    s = prepare(case, seed)
    R, M, op = case["R"], case["M"], case["op"]
    if op == "layernorm":
        h = torch.zeros((M, case["N"]), dtype=torch.float64, device="cuda")
        for r in range(R):
            h += s["x"][r].double()
        if s["res"] is not None:
            h += s["res"].double()
        y = h - h.sum(1, keepdim=True) / case["N"]
        y /= torch.sqrt((y ** 2).sum(1, keepdim=True) / case["N"] + EPS)
        y *= s["gamma"].double()
        if s["bias"] is not None:
            y += s["bias"].double()
        return {"y": y, "h": h} if case["residual_out"] else {"y": y}
    if op == "layernorm_backward":
        N = case["N"]
        dy = torch.zeros((M, N), dtype=torch.float64, device="cuda")
        for r in range(R):
            dy += s["dy"][r].double()
        x = s["h"].double()
        x -= x.sum(1, keepdim=True) / N
        std = torch.sqrt((x ** 2).sum(1, keepdim=True) / N + EPS)
        x /= std
        out = {"dgamma": (dy * x).sum(0)}
        if case["beta"]:
            out["dbeta"] = dy.sum(0)
        dy *= s["gamma"].double()
        dh = (dy - (dy.sum(1, keepdim=True) + x * (dy * x).sum(1, keepdim=True)) / N) / std
        if s["d_res"] is not None:
            dh += s["d_res"].double()
        return {"dh": dh, **out}
    if op.startswith("embedding"):
        N, V = case["N"], R * case["Vs"]
        ids = s["ids"].long()
        there = torch.nonzero((ids >= 0) & (ids < V))[:, 0]
        if op == "embedding":
            out = torch.zeros((M, N), dtype=torch.float64, device="cuda")
            out[there] = s["table"].flatten(0, 1)[ids[there]].double() * case["scale"]
            return out
        d = torch.zeros((V, N), dtype=torch.float64, device="cuda")
        d.index_put_((ids[there],), s["dy"][there].double(), accumulate=True)
        return d.mul_(case["scale"]).view(R, case["Vs"], N)
    K, V, vocab = case["K"], R * case["Vs"], case["vocab"]
    if M * vocab * K * (8 if op == "loss_step" else 2) > 2e13:
        return None
    h, w = s["h"].double(), s["w"].flatten(0, 1).double()
    z = torch.mm(h, w[:vocab].t())
    lse = torch.logsumexp(z, 1)
    targets = s["targets"].long()
    rows = torch.nonzero((targets >= 0) & (targets < vocab))[:, 0]
    loss = torch.zeros(M, dtype=torch.float64, device="cuda")
    loss[rows] = lse[rows] - z[rows, targets[rows]]
    out = {"loss": loss, "lse": lse}
    if op == "loss_step":
        z = torch.exp(z.sub_(lse[:, None]))
        z[rows, targets[rows]] -= 1
        scale = torch.zeros(M, dtype=torch.float64, device="cuda")
        scale[rows] = s["dloss"][rows].double()
        z *= scale[:, None]
        dw = torch.zeros((V, K), dtype=torch.float64, device="cuda")
        dw[:vocab] = torch.mm(z.t(), h)
        out.update(dh=torch.mm(z, w[:vocab]), dw=dw.view(R, case["Vs"], K))
    return out
