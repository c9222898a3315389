"""More operators around a sharded step, measured: the norm of a layer's rows with its
gradient, and the step of a layer's matrices by an orthogonalised momentum: the momentum
of a shard, the orthogonalisation of whole matrices by Newton-Schulz products, and the
update of the shard's master copy and bf16 slot.

M rows of N columns go through a norm; R x C is a matrix to orthogonalise, B of them in
one call; n is a shard's number of elements. ``run`` computes the plain form in 32 bits
with elementary torch operations, or, where ``own`` is true, calls the package.
"""
import math

import torch

own = False

EPS = 1e-5                              # of a norm
TINY = 1e-7                             # of an orthogonalisation
COEF = (3.4445, -4.7750, 2.0315)        # X <- a X + (b A + c A A) X, A = X X^T
MU = 0.95                               # of a momentum
LR, DECAY = 2e-3, 0.1                   # of an update


def _norm(name, op, M, N, **kw):
    c = {"name": name, "op": op, "M": M, "N": N, "kind": "layer", "x": "bf16", "state": "bf16", "out": "bf16",
         "bias": True, "residual": False, "stats": True, "accumulate": False, "grad": "bf16", "wide": False}
    c.update(kw)
    return c


def _orth(name, B, R, C, **kw):
    c = {"name": name, "op": "orthogonalize", "B": B, "R": R, "C": C, "x": "bf16", "steps": 5, "scale": 1.0,
         "wide": False}
    c.update(kw)
    return c


def _flat(name, op, n, **kw):
    return {"name": name, "op": op, "n": n, **kw}


def listed():
    return [
        # one token of GPT-2 small through a layer norm: the smallest call, where latency counts
        _norm("norm-token", "norm_forward", 1, 768, stats=False),
        # GPT-2 small's second norm over 8 sequences of 1,024 tokens, the attention's output
        # added to the residual stream on the way
        _norm("norm-gpt2", "norm_forward", 8192, 768, residual=True),
        # the norm of a Llama-7B shaped block over 8,192 tokens, its residual stream kept in f32
        _norm("norm-llama", "norm_forward", 8192, 4096, kind="rms", bias=False, residual=True, state="f32"),
        # the gradient of a layer norm of an odd width over an odd number of tokens, in f32,
        # added to what earlier micro-batches left
        _norm("norm-grad-odd", "norm_grad", 1023, 1001, x="f32", state="f32", out="f32", grad="f32",
              accumulate=True, wide=True),
        # back through a Llama-7B shaped block's norm, the weight's gradient into an f32 buffer
        _norm("norm-grad-llama", "norm_grad", 8192, 4096, kind="rms", bias=False, residual=True, state="f32",
              grad="f32"),
        # one attention output projection of GPT-2 small: few tiles, where launches count
        _orth("orth-proj", 1, 768, 768),
        # the 12 qkv matrices of GPT-2 small in one call
        _orth("orth-qkv", 12, 768, 2304),
        # a Llama-7B shaped down projection, taller than wide, from an f32 momentum
        _orth("orth-ffn", 1, 11008, 4096, x="f32", scale=0.2 * math.sqrt(11008)),
        # the momentum of one of 8 shards of GPT-2 small
        _flat("momentum-gpt2", "momentum", 15555072, grad="f32", out="bf16"),
        # the momentum of a Llama-7B shaped layer's matrices
        _flat("momentum-llama", "momentum", 4 * 4096 * 4096 + 3 * 4096 * 11008, grad="f32", out="bf16"),
        # the update of the shard of GPT-2 small
        _flat("update-gpt2", "update", 15555072),
        # the update of the Llama-7B shaped layer's matrices
        _flat("update-llama", "update", 4 * 4096 * 4096 + 3 * 4096 * 11008),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, lo, hi):
    n = _log(rng, lo, hi)
    kind = rng.random()
    return max(64, n // 64 * 64) if kind < 0.5 else max(8, n // 8 * 8) if kind < 0.7 else n


def draw(rng):
    op = rng.choice(("norm_forward", "norm_forward", "norm_grad", "norm_grad", "orthogonalize", "orthogonalize",
                     "momentum", "update"))
    ty = ("bf16", "f32")
    if op == "orthogonalize":
        R, C = _width(rng, 64, 11008), _width(rng, 64, 11008)
        if R * C > 11008 * 4096:
            R = 11008 * 4096 // C
        small = min(R, C) ** 2 * (3 * max(R, C) + min(R, C))
        B = max(1, min(_log(rng, 1, 24), int(4096 ** 2 * (3 * 11008 + 4096) // small), 11008 * 8192 // (R * C)))
        return {"op": op, "B": B, "R": R, "C": C, "x": rng.choice(ty), "steps": rng.choice((3, 5, 5, 6)),
                "scale": rng.choice((1.0, 0.2 * math.sqrt(max(R, C)))), "wide": rng.random() < 0.25}
    if op == "momentum":
        return {"op": op, "n": _log(rng, 1 << 12, 1 << 27), "grad": rng.choice(ty), "out": rng.choice(ty)}
    if op == "update":
        return {"op": op, "n": _log(rng, 1 << 12, 1 << 27)}
    M, N = _log(rng, 1, 16384), _width(rng, 64, 16384)
    M = max(1, min(M, 16384 * 4096 // N))
    kind = rng.choice(("layer", "rms"))
    grad = op == "norm_grad"
    return {"op": op, "M": M, "N": N, "kind": kind, "x": rng.choice(ty), "state": rng.choice(ty),
            "out": rng.choice(ty), "bias": kind == "layer", "residual": rng.random() < 0.5,
            "stats": grad or rng.random() < 0.5, "accumulate": grad and rng.random() < 0.5, "grad": rng.choice(ty),
            "wide": rng.random() < 0.25}


_TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}


def prepare(case, seed):
    c = case
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 29)
    s = {"case": c}

    def normal(*shape, scale=1.0):
        return torch.randn(*shape, generator=gen, device=dev) * scale

    if c["op"] in ("momentum", "update"):
        n = c["n"]
        if c["op"] == "momentum":
            s["g"] = normal(n, scale=1e-3).to(_TYPES[c["grad"]])
            s["m"] = normal(n, scale=3e-3)
            return s
        s["p"] = normal(n, scale=0.02)
        s["o"] = normal(n, scale=1 / 64).to(torch.bfloat16)
        s["slot"] = torch.zeros(n, dtype=torch.bfloat16, device=dev)
        return s

    if c["op"] == "orthogonalize":
        # a momentum: a few strong directions that fall off, over noise
        B, R, C = c["B"], c["R"], c["C"]
        k = min(R, C, 32)
        fall = torch.exp(-torch.arange(k, device=dev, dtype=torch.float32) / 6)
        x = torch.matmul(normal(B, R, k) * fall, normal(B, k, C)) + normal(B, R, C, scale=0.3)
        x = (x * 1e-3).to(_TYPES[c["x"]])
        if c["wide"]:
            # columns of rows that hold more beside them
            full = torch.zeros(B, R, (C + 7) // 8 * 8 + 64, dtype=x.dtype, device=dev)
            full[:, :, :C] = x
            x = full[:, :, :C]
        s["x"] = x if B > 1 else x[0]
        return s

    M, N = c["M"], c["N"]

    def rows(dtype, scale=1.0, channels=None):
        # "wide": columns of rows that hold more beside them
        full = normal(M, (N + 7) // 8 * 8 + 64 if c["wide"] else N, scale=scale)
        if channels is not None:
            full[:, :N] = full[:, :N] * channels[0] + channels[1]
        return full.to(_TYPES[dtype])[:, :N]

    # a residual stream: channels of their own size and mean, a few of them large
    size = torch.exp(normal(N, scale=0.5))
    size = torch.where(torch.rand(N, generator=gen, device=dev) < 0.01, size * 10, size)
    stream = (size, normal(N, scale=0.2))
    s["w"] = (1 + normal(N, scale=0.2)).to(torch.bfloat16)
    s["b"] = normal(N, scale=0.1).to(torch.bfloat16) if c["bias"] else None
    if c["op"] == "norm_forward":
        s["x"] = rows(c["x"], 0.5, None if c["residual"] else stream)
        s["residual"] = rows(c["state"], 1.0, stream) if c["residual"] else None
        return s
    s["x"] = rows(c["state"], 1.0, stream)
    s["dy"] = rows(c["x"], 1e-3)
    s["dres"] = rows(c["out"], 1e-3) if c["residual"] else None
    x = s["x"].double()
    mean = x.mean(1) if c["kind"] == "layer" else torch.zeros(M, dtype=torch.float64, device=dev)
    rstd = torch.rsqrt((x - mean[:, None]).square().mean(1) + EPS)
    s["stats"] = torch.stack((mean, rstd), 1).float()       # as the forward pass left them
    # what earlier micro-batches have left, or what the call overwrites
    s["dw"] = normal(N, scale=1e-2).to(_TYPES[c["grad"]])
    s["db"] = normal(N, scale=1e-2).to(_TYPES[c["grad"]]) if c["bias"] else None
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------


def _plain_norm(s):
    c = s["case"]
    got = {}
    x = s["x"].float()
    if s["residual"] is not None:
        got["sum"] = (s["residual"].float() + x).to(_TYPES[c["state"]])
        x = got["sum"].float()              # what is stored is what is normed
    mean = x.mean(1, keepdim=True) if c["kind"] == "layer" else torch.zeros_like(x[:, :1])
    d = x - mean
    rstd = torch.rsqrt(d.square().mean(1, keepdim=True) + EPS)
    y = d * rstd * s["w"].float()
    if s["b"] is not None:
        y = y + s["b"].float()
    got["y"] = y.to(_TYPES[c["out"]])
    if c["stats"]:
        got["stats"] = torch.cat((mean, rstd), 1)
    return got


def _plain_norm_grad(s):
    c = s["case"]
    mean, rstd = s["stats"][:, :1], s["stats"][:, 1:]
    dy = s["dy"].float()
    xhat = (s["x"].float() - mean) * rstd
    g = dy * s["w"].float()
    d = g - xhat * (g * xhat).mean(1, keepdim=True)
    if c["kind"] == "layer":
        d = d - g.mean(1, keepdim=True)
    dx = d * rstd
    if s["dres"] is not None:
        dx = s["dres"].float() + dx
    dw = (dy * xhat).sum(0)
    s["dw"].copy_(s["dw"].float() + dw if c["accumulate"] else dw)
    got = {"dx": dx.to(_TYPES[c["out"]]), "dw": s["dw"]}
    if s["db"] is not None:
        db = dy.sum(0)
        s["db"].copy_(s["db"].float() + db if c["accumulate"] else db)
        got["db"] = s["db"]
    return got


def _plain_orthogonalize(s):
    c = s["case"]
    tall = c["R"] > c["C"]
    x = s["x"].float()
    x = x.transpose(-2, -1).contiguous() if tall else x
    x = x / (x.square().sum((-2, -1), keepdim=True).sqrt() + TINY)
    for _ in range(c["steps"]):
        a = torch.matmul(x, x.transpose(-2, -1).contiguous())
        b = COEF[1] * a + COEF[2] * torch.matmul(a, a)
        x = COEF[0] * x + torch.matmul(b, x)
    x = (x * c["scale"]).to(torch.bfloat16)
    return {"o": x.transpose(-2, -1).contiguous() if tall else x}


def _plain_momentum(s):
    g = s["g"].float()
    s["m"].mul_(MU).add_(g)
    return {"m": s["m"], "u": (g + MU * s["m"]).to(_TYPES[s["case"]["out"]])}


def _plain_update(s):
    s["p"].copy_(s["p"] * (1.0 - LR * DECAY) - LR * s["o"].float())
    s["slot"].copy_(s["p"])
    return {"p": s["p"], "slot": s["slot"]}


_PLAIN = {"norm_forward": _plain_norm, "norm_grad": _plain_norm_grad, "orthogonalize": _plain_orthogonalize,
          "momentum": _plain_momentum, "update": _plain_update}


# ---------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------


def _own(s):
    import zero_partitioned_optimizer_amd as Z
    c = s["case"]
    op = c["op"]
    if op == "orthogonalize":
        return {"o": Z.zero_orthogonalize(s["x"], steps=c["steps"], coefficients=COEF, eps=TINY, scale=c["scale"])}
    if op == "momentum":
        return {"m": s["m"], "u": Z.zero_muon_momentum(s["g"], s["m"], mu=MU, nesterov=True, dtype=_TYPES[c["out"]])}
    if op == "update":
        Z.zero_muon_update(s["p"], s["o"], lr=LR, weight_decay=DECAY, slot=s["slot"])
        return {"p": s["p"], "slot": s["slot"]}
    kind = Z.ZERO_NORM_LAYER if c["kind"] == "layer" else Z.ZERO_NORM_RMS
    if op == "norm_grad":
        dx = Z.zero_norm_grad(s["dy"], s["x"], s["w"], s["stats"], kind=kind, residual_grad=s["dres"],
                              dtype=_TYPES[c["out"]], dweight=s["dw"], dbias=s["db"], accumulate=c["accumulate"])
        got = {"dx": dx, "dw": s["dw"]}
        return got if s["db"] is None else {**got, "db": s["db"]}
    got = Z.zero_norm_forward(s["x"], s["w"], s["b"], kind=kind, eps=EPS, residual=s["residual"],
                              stats=c["stats"], dtype=_TYPES[c["out"]])
    names = ["y"] + (["sum"] if c["residual"] else []) + (["stats"] if c["stats"] else [])
    return dict(zip(names, got)) if len(names) > 1 else {"y": got}


def run(state):
    return _own(state) if own else _PLAIN[state["case"]["op"]](state)


def work(case):
    c = case
    size = {"bf16": 2, "f32": 4}
    if c["op"] == "momentum":
        return {"bytes": c["n"] * (8 + size[c["grad"]] + size[c["out"]]), "flops": 4 * c["n"]}
    if c["op"] == "update":
        return {"bytes": c["n"] * (8 + 2 + 2), "flops": 3 * c["n"]}
    if c["op"] == "orthogonalize":
        m, n = min(c["R"], c["C"]), max(c["R"], c["C"])
        # of the two symmetric products one triangle each
        return {"bytes": c["B"] * m * n * (size[c["x"]] + 2),
                "flops": c["B"] * c["steps"] * (m * (m + 1) * n + m * (m + 1) * m + 2 * m * m * n)}
    M, N = c["M"], c["N"]
    if c["op"] == "norm_forward":
        b = M * N * (size[c["x"]] + size[c["out"]] + (2 * size[c["state"]] if c["residual"] else 0))
        return {"bytes": b + N * (4 if c["bias"] else 2) + (8 * M if c["stats"] else 0), "flops": 8 * M * N}
    b = M * N * (size[c["x"]] + size[c["state"]] + size[c["out"]] * (2 if c["residual"] else 1)) + 2 * N + 8 * M
    return {"bytes": b + N * size[c["grad"]] * (2 if c["bias"] else 1) * (2 if c["accumulate"] else 1),
            "flops": 14 * M * N}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], s["case"]["op"]
    if op == "momentum":
        g = s["g"].double()
        m = MU * s["m"].double() + g
        return {"m": m, "u": MU * m + g}
    if op == "update":
        p = (1 - LR * DECAY) * s["p"].double() - LR * s["o"].double()
        return {"p": p, "slot": p}
    if op == "orthogonalize":
        # the polynomial on the side where the product of the matrix with itself is small
        x = s["x"].double().reshape(c["B"], c["R"], c["C"])
        x = x / (torch.linalg.vector_norm(x, dim=(1, 2), keepdim=True) + TINY)
        eye = torch.eye(min(c["R"], c["C"]), dtype=torch.float64, device=x.device)
        for _ in range(c["steps"]):
            t = x.transpose(1, 2).contiguous()
            gram = torch.bmm(t, x) if c["R"] > c["C"] else torch.bmm(x, t)
            p = torch.bmm(gram, COEF[1] * eye + COEF[2] * gram) + COEF[0] * eye
            x = torch.bmm(x, p) if c["R"] > c["C"] else torch.bmm(p, x)
        x = x * c["scale"]
        return {"o": x if c["B"] > 1 else x[0]}
    N = c["N"]
    w = s["w"].double()
    if op == "norm_forward":
        got = {}
        x = s["x"].double()
        if c["residual"]:
            got["sum"] = x + s["residual"].double()
            x = got["sum"].to(_TYPES[c["state"]]).double()
        mu = x.sum(1) / N if c["kind"] == "layer" else torch.zeros_like(x[:, 0])
        var = ((x - mu[:, None]) ** 2).sum(1) / N
        r = (var + EPS) ** -0.5
        got["y"] = (x - mu[:, None]) * (r[:, None] * w[None]) + (s["b"].double() if c["bias"] else 0.0)
        if c["stats"]:
            got["stats"] = torch.stack((mu, r), 1)
        return got
    # the vector-Jacobian product of y = (x - mean) rstd w, by its two projections
    mu, r = s["stats"].double().unbind(1)
    dy = s["dy"].double()
    h = (s["x"].double() - mu[:, None]) * r[:, None]
    v = dy * w
    dx = v - h * ((v * h).sum(1, keepdim=True) / N)
    if c["kind"] == "layer":
        dx -= v.sum(1, keepdim=True) / N
    dx *= r[:, None]
    got = {"dx": dx + s["dres"].double() if c["residual"] else dx, "dw": (dy * h).sum(0)}
    if c["bias"]:
        got["db"] = dy.sum(0)
    if c["accumulate"]:
        got["dw"] = got["dw"] + s["dw"].double()
        if c["bias"]:
            got["db"] = got["db"] + s["db"].double()
    return got
