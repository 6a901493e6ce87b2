"""Cases of the quantised and backward operators around the all-reduce epilogue.

Four operators:

* ``quant_groups``: all-reduce of R bf16 partials, residual add and RMSNorm with
  FP8 E4M3 codes and one scale per group of columns (fp32, or a power of two);
* ``backward``: the backward pass of all-reduce + residual + RMSNorm, whose
  output gradient arrives as R bf16 partials;
* ``qweight``: the row-parallel linear of a few tokens with 4-bit weights and
  group scales, summed over R ranks;
* ``qweight_qx``: the same with tokens in FP8 codes and group scales, as
  ``quant_groups`` writes them.

``run`` computes them with elementary torch operations in 32 bits, or, where
``own`` is true, with the calls of ``all_reduce_epilogue_gb300``.
"""
import math

import torch

own = False
EPS = 1e-6

_workspace = None


def listed():
    return [
        # the norm after a row-parallel linear, one token, 8 ranks: the smallest decode call
        {"name": "quant token R8", "op": "quant_groups", "R": 8, "M": 1, "N": 7168, "group": 128, "pow2": False,
         "residual": True, "residual_out": True},
        # a ragged decode batch with power-of-two scales per 32 columns, the last group cut short
        {"name": "quant batch R4 pow2", "op": "quant_groups", "R": 4, "M": 37, "N": 4104, "group": 32, "pow2": True,
         "residual": True, "residual_out": True},
        # a prompt of 4096 tokens, 8 ranks
        {"name": "quant prompt R8", "op": "quant_groups", "R": 8, "M": 4096, "N": 7168, "group": 128, "pow2": False,
         "residual": True, "residual_out": True},
        # a short fine-tuning step, one rank, the gradient of the residual stream present
        {"name": "backward short R1", "op": "backward", "R": 1, "M": 64, "N": 4096, "dres": True},
        # odd row count, width no multiple of a tile, the last layer (no residual gradient)
        {"name": "backward odd R3", "op": "backward", "R": 3, "M": 1001, "N": 5000, "dres": False},
        # a training step's full batch on one rank and on eight
        {"name": "backward batch R1", "op": "backward", "R": 1, "M": 16384, "N": 4096, "dres": True},
        {"name": "backward batch R8", "op": "backward", "R": 8, "M": 4096, "N": 7168, "dres": True},
        # the smallest product: one token, a tiny layer on two ranks
        {"name": "qweight tiny", "op": "qweight", "R": 2, "M": 1, "N": 256, "K": 128, "group": 128, "zero": True},
        # one token through a row-parallel layer of 8 ranks
        {"name": "qweight token R8", "op": "qweight", "R": 8, "M": 1, "N": 7168, "K": 2048, "group": 128,
         "zero": True},
        # a decode batch through a large layer, symmetric weights in groups of 64
        {"name": "qweight batch R8", "op": "qweight", "R": 8, "M": 16, "N": 8192, "K": 4096, "group": 64,
         "zero": False},
        # a few tokens in 8 bits
        {"name": "qweight_qx few R4", "op": "qweight_qx", "R": 4, "M": 5, "N": 4096, "K": 2048, "group": 128,
         "zero": True, "xgroup": 128, "pow2": False},
        # a wide decode batch in 8 bits with power-of-two scales
        {"name": "qweight_qx batch R8", "op": "qweight_qx", "R": 8, "M": 64, "N": 7168, "K": 2048, "group": 128,
         "zero": False, "xgroup": 32, "pow2": True},
    ]


def _log(rng, lo, hi, step=1):
    """A multiple of ``step`` in [lo, hi], spread over the logarithm."""
    v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + step))))
    return max(lo, min(hi, v // step * step))


def draw(rng):
    op = rng.choice(["quant_groups", "backward", "qweight", "qweight_qx"])
    R = rng.randint(1, 8)
    if op == "quant_groups":
        N = _log(rng, 64, 8192, 8)
        M = _log(rng, 1, min(8192, max(1, 8 * 4096 * 7168 // (R * N))))
        return {"op": op, "R": R, "M": M, "N": N, "group": rng.choice([32, 64, 128]), "pow2": rng.random() < 0.5,
                "residual": rng.random() < 0.8, "residual_out": rng.random() < 0.8}
    if op == "backward":
        N = _log(rng, 64, 16384, 8)
        M = _log(rng, 1, min(16384, max(1, 8 * 4096 * 7168 // ((R + 2) * N))))
        return {"op": op, "R": R, "M": M, "N": N, "dres": rng.random() < 0.7}
    c = {"op": op, "R": R, "M": _log(rng, 1, 64), "N": _log(rng, 64, 8192, 8), "K": _log(rng, 64, 4096, 32),
         "group": rng.choice([32, 64, 128]), "zero": rng.random() < 0.5}
    if op == "qweight_qx":
        c.update(xgroup=rng.choice([32, 64, 128]), pow2=rng.random() < 0.5)
    return c


def _groups(n, g):
    return -(-n // g)


def prepare(case, seed):
    global _workspace
    gen = torch.Generator(device="cuda").manual_seed(seed)
    R, M, N = case["R"], case["M"], case["N"]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale)

    def channels(n):
        """Per-channel magnitudes: most near one, a few outlier channels."""
        c = torch.exp(normal(n, scale=0.4))
        return torch.where(torch.rand(n, generator=gen, device="cuda") < 0.004, c * 20, c)

    s = dict(case)
    if case["op"] == "quant_groups":
        x = torch.empty((R, M, N), dtype=torch.bfloat16, device="cuda")
        ch = channels(N)
        for r in range(R):
            x[r] = normal(M, N) * ch
        res = (normal(M, N) * ch * 2).to(torch.bfloat16) if case["residual"] else None
        if M > 8:  # rows that pad a batch
            x[:, -2:] = 0
            if res is not None:
                res[-2:] = 0
        sdt = torch.uint8 if case["pow2"] else torch.float32
        s.update(x=x, partials=list(x), res=res, gamma=1 + normal(N, scale=0.1),
                 out_q=torch.empty((M, N), dtype=torch.uint8, device="cuda"),
                 out_scale=torch.empty((M, _groups(N, case["group"])), dtype=sdt, device="cuda"),
                 res_out=torch.empty((M, N), dtype=torch.bfloat16, device="cuda") if case["residual_out"] else None)
    elif case["op"] == "backward":
        dy = torch.empty((R, M, N), dtype=torch.bfloat16, device="cuda")
        for r in range(R):
            dy[r] = normal(M, N, scale=1e-2)
        if M > 8:  # rows that take no part in the loss
            dy[:, M // 2] = 0
        s.update(dy=dy, partials=list(dy), h=(normal(M, N) * channels(N) * 3).to(torch.bfloat16),
                 gamma=1 + normal(N, scale=0.1),
                 d_res=normal(M, N, scale=1e-2).to(torch.bfloat16) if case["dres"] else None,
                 dh=torch.empty((M, N), dtype=torch.bfloat16, device="cuda"),
                 dgamma=torch.empty(N, dtype=torch.float32, device="cuda"))
    else:
        K, G = case["K"], _groups(case["K"], case["group"])
        codes = torch.randint(0, 256, (R, N, K // 2), generator=gen, device="cuda", dtype=torch.uint8)
        scale = (torch.exp(normal(R, N, G, scale=0.3)) * (0.2 / math.sqrt(R * K))).to(torch.bfloat16)
        zero = torch.randint(5, 12, (R, N, G), generator=gen, device="cuda", dtype=torch.uint8) if case["zero"] else None
        x = normal(R, M, K) * channels(K)
        s.update(codes=codes, scale=scale, zero=zero, out=torch.empty((M, N), dtype=torch.bfloat16, device="cuda"))
        if case["op"] == "qweight":
            s["x"] = x.to(torch.bfloat16)
            s["tokens"] = list(s["x"])
        else:
            g = case["xgroup"]
            xg = _pad(x, g).unflatten(-1, (-1, g))
            s["xscale"], sf = _scales(xg.abs().amax(-1), case["pow2"])
            s["xq"] = (xg / sf[..., None]).flatten(-2)[..., :K].to(torch.float8_e4m3fn).view(torch.uint8).contiguous()
            s["tokens"], s["token_scales"] = list(s["xq"]), list(s["xscale"])
    if own:
        import all_reduce_epilogue_gb300 as are
        if _workspace is None:  # one workspace for the program
            _workspace = are.Workspace(R_max=8, M_max=1, N_max=16384)
        s["ws"] = _workspace
        if "codes" in s:
            s["w"] = [are.QWeight(codes[r], scale[r], None if zero is None else zero[r], case["group"])
                      for r in range(R)]
    return s


def _pad(t, g):
    """The last axis filled up with zeros to a multiple of g."""
    n = t.shape[-1]
    return t if n % g == 0 else torch.nn.functional.pad(t, (0, g - n % g))


def _scales(amax, pow2):
    """(the scales as stored, as fp32) of groups with these largest magnitudes: amax / 448, or the smallest
    power of two that brings the group to 448 or less; one for a group of zeros."""
    if not pow2:
        f = torch.where(amax > 0, amax / 448, torch.ones_like(amax))
        return f, f
    m, e = torch.frexp(amax)  # amax = m * 2^e, 0.5 <= m < 1; 448 = 0.875 * 2^9
    e = torch.where(amax > 0, e - 9 + (m > 0.875), torch.zeros_like(e)).clamp(-127, 127)
    return (e + 127).to(torch.uint8), torch.ldexp(torch.ones_like(amax), e)


def _dequant(codes, scale, zero, group):
    """fp32 [..., N, K] of 4-bit codes, the lower four bits first."""
    u = torch.stack((codes & 15, codes >> 4), -1).flatten(-2).float()
    K = u.shape[-1]
    z = 8.0 if zero is None else zero.float().repeat_interleave(group, -1)[..., :K]
    return (u - z) * scale.float().repeat_interleave(group, -1)[..., :K]


def run(s):
    if own:
        return _run_own(s)
    op = s["op"]
    if op == "quant_groups":
        h = s["x"].float().sum(0)
        if s["res"] is not None:
            h = h + s["res"].float()
        y = h * torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS) * s["gamma"]
        yg = _pad(y, s["group"]).unflatten(-1, (-1, s["group"]))
        stored, f = _scales(yg.abs().amax(-1), s["pow2"])
        q = (yg / f[..., None]).flatten(-2)[..., :s["N"]].clamp(-448, 448).to(torch.float8_e4m3fn)
        out = {"q": q, "scale": stored.view(torch.float8_e8m0fnu) if s["pow2"] else stored}
        if s["residual_out"]:
            out["h"] = h.to(torch.bfloat16)
        return out
    if op == "backward":
        dy, h = s["dy"].float().sum(0), s["h"].float()
        inv = torch.rsqrt((h * h).mean(-1, keepdim=True) + EPS)
        xhat, g = h * inv, dy * s["gamma"]
        dh = inv * (g - xhat * (g * xhat).mean(-1, keepdim=True))
        if s["d_res"] is not None:
            dh = dh + s["d_res"].float()
        return {"dh": dh.to(torch.bfloat16), "dgamma": (dy * xhat).sum(0)}
    if op == "qweight":
        x = s["x"].float()
    else:
        f = s["xscale"].view(torch.float8_e8m0fnu).float() if s["pow2"] else s["xscale"]
        x = s["xq"].view(torch.float8_e4m3fn).float() * f.repeat_interleave(s["xgroup"], -1)[..., :s["K"]]
    w = _dequant(s["codes"], s["scale"], s["zero"], s["group"])
    return torch.matmul(x, w.transpose(-1, -2)).sum(0).to(torch.bfloat16)


def _run_own(s):
    import all_reduce_epilogue_gb300 as are
    op = s["op"]
    if op == "quant_groups":
        are.allreduce_rmsnorm_quant_groups(s["partials"], s["res"], s["gamma"], EPS, s["out_q"], s["out_scale"],
                                           s["ws"], group=s["group"], residual_out=s["res_out"])
        out = {"q": s["out_q"].view(torch.float8_e4m3fn),
               "scale": s["out_scale"].view(torch.float8_e8m0fnu) if s["pow2"] else s["out_scale"]}
        if s["residual_out"]:
            out["h"] = s["res_out"]
        return out
    if op == "backward":
        are.allreduce_rmsnorm_backward(s["partials"], s["h"], s["gamma"], EPS, s["dh"], s["dgamma"], s["ws"],
                                       dres=s["d_res"])
        return {"dh": s["dh"], "dgamma": s["dgamma"]}
    if op == "qweight":
        are.gemm_ar_qweight(s["tokens"], s["w"], s["out"], s["ws"])
    else:
        are.gemm_ar_qweight_qx(s["tokens"], s["token_scales"], s["w"], s["out"], s["ws"], xgroup=s["xgroup"])
    return s["out"]


def work(case):
    R, M, N = case["R"], case["M"], case["N"]
    if case["op"] == "quant_groups":
        groups = M * _groups(N, case["group"])
        return {"bytes": M * N * (2 * R + 2 * case["residual"] + 1 + 2 * case["residual_out"]) + 4 * N
                + groups * (1 if case["pow2"] else 4), "flops": M * N * (R + 8)}
    if case["op"] == "backward":
        return {"bytes": M * N * (2 * R + 2 + 2 * case["dres"] + 2) + 8 * N, "flops": M * N * (R + 12)}
    K, G = case["K"], _groups(case["K"], case["group"])
    x = M * K * 2 if case["op"] == "qweight" else M * K + M * _groups(K, case["xgroup"]) * (1 if case["pow2"] else 4)
    return {"bytes": R * (N * K // 2 + N * G * (3 if case["zero"] else 2) + x) + M * N * 2, "flops": 2 * R * M * N * K}


def exact(case, seed):
    """The operators from their definitions in 64 bits."""
    s = prepare(case, seed)
    R, M, N = case["R"], case["M"], case["N"]
    if case["op"] == "quant_groups":
        h = torch.zeros((M, N), dtype=torch.float64, device="cuda")
        for r in range(R):
            h += s["x"][r].double()
        if s["res"] is not None:
            h += s["res"].double()
        y = h / torch.sqrt((h ** 2).sum(1) / N + EPS)[:, None] * s["gamma"].double()
        q, scale = torch.empty_like(y), []
        for a in range(0, N, case["group"]):
            part = y[:, a:a + case["group"]]
            top = part.abs().max(1).values
            f = top / 448
            if case["pow2"]:
                f = torch.exp2(torch.ceil(torch.log2(f)).clamp(-127, 127))
            f = torch.where(top > 0, f, torch.ones_like(f))
            q[:, a:a + case["group"]] = (part / f[:, None]).float().clamp(-448, 448).to(torch.float8_e4m3fn).double()
            scale.append(f)
        out = {"q": q, "scale": torch.stack(scale, 1)}
        if case["residual_out"]:
            out["h"] = h
        return out
    if case["op"] == "backward":
        dy = torch.zeros((M, N), dtype=torch.float64, device="cuda")
        for r in range(R):
            dy += s["dy"][r].double()
        h, gamma = s["h"].double(), s["gamma"].double()
        rms = torch.sqrt((h ** 2).sum(1) / N + EPS)[:, None]
        dgamma = (dy * h / rms).sum(0)
        dy *= gamma
        dh = dy / rms - h * ((dy * h).sum(1)[:, None] / (N * rms ** 3))
        if s["d_res"] is not None:
            dh += s["d_res"].double()
        return {"dh": dh, "dgamma": dgamma}
    K, group = case["K"], case["group"]
    y = torch.zeros((M, N), dtype=torch.float64, device="cuda")
    for r in range(R):
        c = s["codes"][r].long()
        w = torch.empty((N, K), dtype=torch.float64, device="cuda")
        w[:, 0::2], w[:, 1::2] = (c % 16).double(), torch.div(c, 16, rounding_mode="floor").double()
        x = (s["x"][r] if case["op"] == "qweight" else s["xq"][r].view(torch.float8_e4m3fn)).double()
        for i, a in enumerate(range(0, K, group)):
            z = 8.0 if s["zero"] is None else s["zero"][r, :, i:i + 1].double()
            w[:, a:a + group] = (w[:, a:a + group] - z) * s["scale"][r, :, i:i + 1].double()
        if case["op"] == "qweight_qx":
            for i, a in enumerate(range(0, K, case["xgroup"])):
                f = s["xscale"][r, :, i:i + 1].double()
                x[:, a:a + case["xgroup"]] *= torch.exp2(f - 127) if case["pow2"] else f
        y += x @ w.T
    return y
