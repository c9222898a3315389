"""The layer operators around a sharded step, measured: a linear layer's product with
its epilogue, its gradients by input and by weight, and dropout with its gradient.

M is the number of rows (tokens), K a layer's inputs,
N its outputs. Activations and weights are bf16; what leaves an operator is bf16 or f32.
Weights lie as [N, K] ("oi") or [K, N] ("io"). ``run`` computes the plain form in 32
bits with elementary torch operations, or, where ``own`` is true, calls the package.
"""
import math

import torch

own = False

ACTS = ("none", "relu", "gelu", "silu")
LARGEST = 8192 * 4096 * 11008           # M * N * K of the largest product


def _case(name, op, M, K=0, N=0, **kw):
    c = {"name": name, "op": op, "M": M, "K": K, "N": N, "layout": "oi", "bias": False, "act": "none",
         "preact": False, "p": 0.0, "residual": False, "out": "bf16", "accumulate": False, "wide": False}
    c.update(kw)
    return c


def listed():
    return [
        # one token through a GPT-2 small qkv layer: the smallest call, where latency counts
        _case("forward-token", "forward", 1, 768, 2304, bias=True),
        # the attention output projection of GPT-2 small over 8 sequences of 1,024 tokens,
        # with the bias, dropout and residual of its block in the epilogue
        _case("forward-proj", "forward", 8192, 768, 768, layout="io", bias=True, p=0.1, residual=True),
        # the gate layer of a Llama-7B shaped block over 8,192 tokens, its pre-activation kept
        _case("forward-ffn", "forward", 8192, 4096, 11008, act="silu", preact=True),
        # logits of one sequence over GPT-2 small's vocabulary: an odd width, f32 out
        _case("forward-head", "forward", 1023, 768, 50257, out="f32"),
        # the gradient back through that head: rows of an odd length are summed over
        _case("grad-input-head", "grad_input", 1023, 768, 50257),
        # back through a Llama-7B shaped down projection, into the activation below it
        _case("grad-input-ffn", "grad_input", 8192, 11008, 4096, act="silu"),
        # the projection's weight and bias gradient, added to what earlier micro-batches left
        _case("grad-weight-proj", "grad_weight", 8192, 768, 768, layout="io", bias=True, accumulate=True),
        # a Llama-7B shaped weight gradient into an f32 gradient buffer
        _case("grad-weight-ffn", "grad_weight", 8192, 4096, 11008, out="f32", accumulate=True),
        # dropout and residual over the hidden states of 8 sequences of 1,024 tokens
        _case("dropout-add", "dropout_add", 8192, 0, 768, p=0.1, residual=True),
        # dropout over the wide inner states of a long batch kept in f32
        _case("dropout-wide", "dropout_add", 16384, 0, 11008, p=0.2, out="f32"),
        # the gradient of dropout alone over one sequence of 128 tokens
        _case("dropout-grad-small", "dropout_grad", 128, 0, 768, p=0.1),
        # the gradient of dropout and activation over the inner states of 8,192 tokens
        _case("dropout-grad-gelu", "dropout_grad", 8192, 0, 11008, p=0.1, act="gelu"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng, hi):
    n = _log(rng, 64, hi)
    kind = rng.random()
    return max(64, n // 64 * 64) if kind < 0.5 else max(64, n // 8 * 8) if kind < 0.7 else n


def draw(rng):
    op = rng.choice(("forward", "forward", "grad_input", "grad_input", "grad_weight", "grad_weight",
                     "dropout_add", "dropout_grad"))
    M = _log(rng, 1, 16384)
    K, N = _width(rng, 11008), _width(rng, 50257 if rng.random() < 0.15 else 11008)
    if op.startswith("dropout"):
        K = 0
        M = min(M, 16384 * 11008 // N)
    else:
        M = max(1, min(M, LARGEST // (K * N), 16384 * 11008 // max(K, N)))
    p = rng.choice((0.0, 0.1, 0.25, 0.5))
    c = {"op": op, "M": M, "K": K, "N": N, "layout": "oi", "bias": False, "act": "none",
         "preact": False, "p": 0.0, "residual": False, "out": rng.choice(("bf16", "f32")),
         "accumulate": False, "wide": rng.random() < 0.25}
    if op in ("forward", "grad_input", "grad_weight"):
        c["layout"] = rng.choice(("oi", "io"))
    if op in ("forward", "grad_input", "dropout_grad"):
        c["act"] = rng.choice(ACTS)
        c["p"] = p
    if op in ("forward", "grad_weight"):
        c["bias"] = rng.random() < 0.5
    if op == "forward":
        c["residual"] = rng.random() < 0.5
        c["preact"] = c["act"] != "none" and rng.random() < 0.5
    if op == "grad_weight":
        c["accumulate"] = rng.random() < 0.5
    if op == "dropout_add":
        c["p"] = max(p, 0.1)
        c["residual"] = rng.random() < 0.5
    if op == "dropout_grad" and c["act"] == "none":
        c["p"] = max(p, 0.1)
    return c


def _dtype(c):
    return torch.float32 if c["out"] == "f32" else torch.bfloat16


def prepare(case, seed):
    c = case
    dev = torch.device("cuda", torch.cuda.current_device())
    gen = torch.Generator(device=dev)
    gen.manual_seed(int(seed) * 7919 + 17)
    op, M, K, N, ty = c["op"], c["M"], c["K"], c["N"], _dtype(c)

    def rows(m, n, scale, dtype=torch.bfloat16):
        # activations; "wide": columns of rows that hold more beside them
        full = torch.randn(m, (n + 7) // 8 * 8 + 64 if c["wide"] else n, generator=gen, device=dev) * scale
        return full.to(dtype)[:, :n]

    def flat(shape, scale, dtype=torch.bfloat16):
        return (torch.randn(*shape, generator=gen, device=dev) * scale).to(dtype)

    s = {"case": c, "seed": int(seed) * 2654435761 + 12345, "offset": int(seed) % 1000}
    wshape = (N, K) if c["layout"] == "oi" else (K, N)
    if op == "forward":
        s["x"] = rows(M, K, 1.0)
        s["w"] = flat(wshape, 0.02)
        s["bias"] = flat((N,), 0.02) if c["bias"] else None
        s["residual"] = rows(M, N, 1.0, ty) if c["residual"] else None
    elif op == "grad_input":
        s["dz"] = rows(M, N, 1e-3)
        s["w"] = flat(wshape, 0.02)
        s["z"] = rows(M, K, 1.0) if c["act"] != "none" else None
    elif op == "grad_weight":
        s["dz"] = rows(M, N, 1e-3)
        s["x"] = rows(M, K, 1.0)
        # what earlier micro-batches have left, or what the call overwrites
        s["dw"] = flat(wshape, 1e-2, ty)
        s["db"] = flat((N,), 1e-2, ty) if c["bias"] else None
    elif op == "dropout_add":
        s["x"] = rows(M, N, 1.0, ty)
        s["residual"] = rows(M, N, 1.0, ty) if c["residual"] else None
    else:
        s["dy"] = rows(M, N, 1e-3, ty)
        s["z"] = rows(M, N, 1.0) if c["act"] != "none" else None
    return s


# ---------------------------------------------------------------------------
# the plain form
# ---------------------------------------------------------------------------

_LOW = 0xFFFFFFFF


def _keep(s, rows, cols, dev):
    """keep[i, j], from Philox4x32-10 with counter (j / 8, i, offset) and the seed as its key:
    16 bits for each of the 8 columns that share a counter."""
    c = s["case"]
    thr = int(round(c["p"] * 65536))
    g = (cols + 7) // 8
    c0 = torch.arange(g, device=dev, dtype=torch.int64)[None, :].expand(rows, g)
    c1 = torch.arange(rows, device=dev, dtype=torch.int64)[:, None].expand(rows, g)
    c2 = torch.full((1, 1), s["offset"] & _LOW, device=dev, dtype=torch.int64).expand(rows, g)
    c3 = torch.full((1, 1), (s["offset"] >> 32) & _LOW, device=dev, dtype=torch.int64).expand(rows, g)
    k0, k1 = s["seed"] & _LOW, (s["seed"] >> 32) & _LOW
    for _ in range(10):
        a, b = c0 * 0xD2511F53, c2 * 0xCD9E8D57
        c0, c1, c2, c3 = ((b >> 32) & _LOW) ^ c1 ^ k0, b & _LOW, ((a >> 32) & _LOW) ^ c3 ^ k1, a & _LOW
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    words = torch.stack((c0, c1, c2, c3), dim=-1)
    halves = torch.stack((words & 0xFFFF, words >> 16), dim=-1)
    return halves.reshape(rows, 8 * g)[:, :cols] >= thr, 65536.0 / (65536 - thr)


def _drop(s, h):
    if s["case"]["p"] == 0.0:
        return h
    keep, scale = _keep(s, h.shape[0], h.shape[1], h.device)
    return torch.where(keep, h * scale, torch.zeros_like(h))


_C, _A = math.sqrt(2.0 / math.pi), 0.044715


def _act(name, z):
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return 0.5 * z * (1 + torch.tanh(_C * (z + _A * z * z * z)))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def _act_grad(name, z):
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        t = torch.tanh(_C * (z + _A * z * z * z))
        return 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * _C * (1 + 3 * _A * z * z)
    if name == "silu":
        g = torch.sigmoid(z)
        return g * (1 + z * (1 - g))
    return torch.ones_like(z)


def _plain(s):
    c = s["case"]
    op, ty = c["op"], _dtype(c)
    if op == "forward":
        w = s["w"].float()
        z = s["x"].float() @ (w.t() if c["layout"] == "oi" else w)
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y = _drop(s, _act(c["act"], z))
        if s["residual"] is not None:
            y = s["residual"].float() + y
        return {"y": y.to(ty), "z": z.to(torch.bfloat16)} if c["preact"] else {"y": y.to(ty)}
    if op == "grad_input":
        w = s["w"].float()
        d = _drop(s, s["dz"].float() @ (w if c["layout"] == "oi" else w.t()))
        if s["z"] is not None:
            d = d * _act_grad(c["act"], s["z"].float())
        return {"dx": d.to(ty)}
    if op == "grad_weight":
        dz, x = s["dz"].float(), s["x"].float()
        dw = dz.t() @ x if c["layout"] == "oi" else x.t() @ dz
        db = dz.sum(0) if c["bias"] else None
        if c["accumulate"]:
            dw = s["dw"].float() + dw
            db = s["db"].float() + db if c["bias"] else None
        s["dw"].copy_(dw)
        if c["bias"]:
            s["db"].copy_(db)
            return {"dw": s["dw"], "db": s["db"]}
        return {"dw": s["dw"]}
    if op == "dropout_add":
        y = _drop(s, s["x"].float())
        return {"y": (y if s["residual"] is None else s["residual"].float() + y).to(ty)}
    d = _drop(s, s["dy"].float())
    if s["z"] is not None:
        d = d * _act_grad(c["act"], s["z"].float())
    return {"dz": d.to(ty)}


# ---------------------------------------------------------------------------
# the package's operators
# ---------------------------------------------------------------------------


def _own(s):
    import zero_partitioned_optimizer_amd as Z
    c = s["case"]
    op, ty = c["op"], _dtype(c)
    lay = Z.ZERO_W_OUT_IN if c["layout"] == "oi" else Z.ZERO_W_IN_OUT
    act = (Z.ZERO_ACT_NONE, Z.ZERO_ACT_RELU, Z.ZERO_ACT_GELU, Z.ZERO_ACT_SILU)[ACTS.index(c["act"])]
    drop = Z.zero_dropout(c["p"], s["seed"], s["offset"]) if c["p"] else None
    if op == "forward":
        got = Z.zero_linear_forward(s["x"], s["w"], s["bias"], w_layout=lay, act=act, dropout=drop,
                                    residual=s["residual"], preact=c["preact"], dtype=ty)
        return {"y": got[0], "z": got[1]} if c["preact"] else {"y": got}
    if op == "grad_input":
        return {"dx": Z.zero_linear_grad_input(s["dz"], s["w"], w_layout=lay, act=act, preact=s["z"],
                                               dropout=drop, dtype=ty)}
    if op == "grad_weight":
        Z.zero_linear_grad_weight(s["dz"], s["x"], s["dw"], s["db"], w_layout=lay,
                                  accumulate=c["accumulate"])
        return {"dw": s["dw"], "db": s["db"]} if c["bias"] else {"dw": s["dw"]}
    if op == "dropout_add":
        return {"y": Z.zero_dropout_add(s["x"], drop, residual=s["residual"])}
    return {"dz": Z.zero_dropout_grad(s["dy"], drop, act=act, preact=s["z"])}


def run(state):
    return _own(state) if own else _plain(state)


def work(case):
    c = case
    M, K, N = c["M"], c["K"], c["N"]
    out = 4 if c["out"] == "f32" else 2
    if c["op"] == "forward":
        b = 2 * (M * K + N * K) + M * N * (out * (2 if c["residual"] else 1) + (2 if c["preact"] else 0))
        return {"bytes": b + (2 * N if c["bias"] else 0), "flops": 2 * M * N * K}
    if c["op"] == "grad_input":
        return {"bytes": 2 * (M * N + N * K) + M * K * (out + (2 if c["act"] != "none" else 0)), "flops": 2 * M * N * K}
    if c["op"] == "grad_weight":
        return {"bytes": 2 * (M * N + M * K) + (N * K + (N if c["bias"] else 0)) * out * (2 if c["accumulate"] else 1),
                "flops": 2 * M * N * K}
    if c["op"] == "dropout_add":
        return {"bytes": M * N * out * (3 if c["residual"] else 2), "flops": 2 * M * N}
    return {"bytes": M * N * (2 * out + (2 if c["act"] != "none" else 0)), "flops": (2 if c["act"] == "none" else 12) * M * N}


# ---------------------------------------------------------------------------
# the definition in 64 bits
# ---------------------------------------------------------------------------


def _exact_factor(s, rows, cols, dev):
    """0 where an element is dropped and the survivors' factor elsewhere, [rows, cols] in 64 bits,
    with the generator written out on the host in unsigned 64-bit integers."""
    import numpy as np
    c = s["case"]
    thr = int(round(c["p"] * 65536))
    u = np.uint64
    low, half = u(_LOW), u(32)
    groups = -(-cols // 8)
    out = np.empty((rows, groups, 8), np.uint16)
    step = max(1, (1 << 20) // groups)
    for r0 in range(0, rows, step):
        r1 = min(rows, r0 + step)
        x = [np.tile(np.arange(groups, dtype=u), r1 - r0), np.repeat(np.arange(r0, r1, dtype=u), groups),
             np.full((r1 - r0) * groups, s["offset"] & _LOW, u), np.full((r1 - r0) * groups, (s["offset"] >> 32) & _LOW, u)]
        key = [s["seed"] & _LOW, (s["seed"] >> 32) & _LOW]
        for _ in range(10):
            m0, m1 = u(0xD2511F53) * x[0], u(0xCD9E8D57) * x[2]
            x = [(m1 >> half) ^ x[1] ^ u(key[0]), m1 & low, (m0 >> half) ^ x[3] ^ u(key[1]), m0 & low]
            key = [(key[0] + 0x9E3779B9) & _LOW, (key[1] + 0xBB67AE85) & _LOW]
        for k in range(4):
            out[r0:r1, :, 2 * k] = (x[k] & u(0xFFFF)).reshape(r1 - r0, groups)
            out[r0:r1, :, 2 * k + 1] = (x[k] >> u(16)).reshape(r1 - r0, groups)
    keep = out.reshape(rows, 8 * groups)[:, :cols] >= thr
    return torch.from_numpy(keep).to(dev).double() / (1.0 - thr / 65536.0)


def _exact_act(name, z):
    """(act(z), act'(z)) in 64 bits from the logistic function."""
    if name == "none":
        return z, torch.ones_like(z)
    if name == "relu":
        on = (z > 0).double()
        return z * on, on
    if name == "silu":
        g = 1 / (1 + torch.exp(-z))
        return z * g, g + z * g * (1 - g)
    a = 2 * math.sqrt(2 / math.pi)
    g = 1 / (1 + torch.exp(-a * (z + 0.044715 * z ** 3)))
    return z * g, g + z * g * (1 - g) * a * (1 + 0.134145 * z ** 2)


def exact(case, seed):
    s = prepare(case, seed)
    c, op = s["case"], s["case"]["op"]
    oi = c["layout"] == "oi"
    if op == "forward":
        w = s["w"].double()
        z = torch.mm(s["x"].double(), w.t().contiguous() if oi else w)
        del w
        if c["bias"]:
            z += s["bias"].double()
        y = _exact_act(c["act"], z)[0]
        if c["p"]:
            y = y * _exact_factor(s, c["M"], c["N"], z.device)
        if c["residual"]:
            y = y + s["residual"].double()
        return {"y": y, "z": z} if c["preact"] else {"y": y}
    if op == "grad_input":
        w = s["w"].double()
        d = torch.mm(s["dz"].double(), w if oi else w.t().contiguous())
        if c["p"]:
            d *= _exact_factor(s, c["M"], c["K"], d.device)
        if c["act"] != "none":
            d *= _exact_act(c["act"], s["z"].double())[1]
        return {"dx": d}
    if op == "grad_weight":
        dz, x = s["dz"].double(), s["x"].double()
        dw = torch.mm(dz.t().contiguous(), x) if oi else torch.mm(x.t().contiguous(), dz)
        got = {"dw": dw + s["dw"].double() if c["accumulate"] else dw}
        if c["bias"]:
            db = dz.sum(0)
            got["db"] = db + s["db"].double() if c["accumulate"] else db
        return got
    if op == "dropout_add":
        y = s["x"].double() * _exact_factor(s, c["M"], c["N"], s["x"].device)
        return {"y": y + s["residual"].double() if c["residual"] else y}
    d = s["dy"].double()
    if c["p"]:
        d = d * _exact_factor(s, c["M"], c["N"], d.device)
    if c["act"] != "none":
        d = d * _exact_act(c["act"], s["z"].double())[1]
    return {"dz": d}
