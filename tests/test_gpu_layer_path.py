"""The layer operators together, as a training program uses them: a layer's tensors
fetched out of the rank shards, forward with dropout, backward into the flat
gradient buffers of two data-parallel ranks, the sharded step on their slices, and
the next pass with the stepped parameters. Gradients are checked against the
formulas in 64 bits and against differences of the loss."""
import numpy as np
import pytest
import torch

import layer_ref as R
import oracle
from gpu_util import dev, say, to_host

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def f64(t):
    return t.detach().cpu().double().numpy()


class Mlp:
    """y = x + D(gelu(x W1 + b1) W2 + b2) over flat buffers (weights [in, out] and
    [out, in])."""

    def __init__(self, Z, d, inner, N):
        self.Z, self.d, self.inner, self.N = Z, d, inner, N
        self.numels = [5, d * inner, inner, inner * d, d]
        h = Z.zero_layout_build(self.numels, N, 8, 8)
        self.offsets, self.S = Z.zero_layout_offsets(h), Z.zero_layout_info_get(h).shard_S
        Z.zero_layout_free(h)
        self.l1 = Z.FlatLinear(self.offsets, self.numels, 1, 2, d, inner, w_layout=Z.ZERO_W_IN_OUT, act=Z.ZERO_ACT_GELU)
        self.l2 = Z.FlatLinear(self.offsets, self.numels, 3, 4, inner, d, w_layout=Z.ZERO_W_OUT_IN)

    def run(self, shards, x, dy, drop, grads, accumulate=False):
        self.l1.fetch(shards, self.S)
        self.l2.fetch(shards, self.S)
        a, z = self.l1.forward(x)
        y, _ = self.l2.forward(a, dropout=drop, residual=x)
        d2 = self.Z.zero_dropout_grad(dy, drop)
        dz = self.l2.backward(d2, a, grads, accumulate=accumulate, below=(self.l1.act, z, None))
        dx = self.l1.backward(dz, x, grads, accumulate=accumulate)
        out = dict(a=a, z=z, y=y, d2=d2, dz=dz, dx=dx)
        self.l1.release(), self.l2.release()
        return out

    def views(self, flat):
        o, d, n = self.offsets, self.d, self.inner
        return (flat[o[1]:o[1] + d * n].reshape(d, n), flat[o[2]:o[2] + n], flat[o[3]:o[3] + n * d].reshape(d, n),
                flat[o[4]:o[4] + d])


def check(name, got, want, err):
    d = np.abs(f64(got) - want)
    assert (d <= err).all(), (name, float(d.max()), float((d - err).max()))


def test_training_steps_of_an_mlp(Z):
    d, inner, M, N = 136, 264, 192, 2
    net = Mlp(Z, d, inner, N)
    rng = np.random.default_rng(21)
    say("mlp path", d, inner, M)
    flat = (rng.standard_normal(N * net.S) * 0.1).astype(np.float32)
    steps = [Z.DeviceShardStep(net.S, N, Z.ZERO_BF16, torch.from_numpy(flat[r * net.S:(r + 1) * net.S]).to(dev()),
                               lr=1e-2, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.01) for r in range(N)]
    grads = [torch.zeros(N * net.S, dtype=BF, device=dev()) for _ in range(N)]
    before = None
    for it in range(2):
        shards = [s.current_slot() for s in steps]
        params = np.concatenate([f64(s.view(BF)) for s in shards])
        if before is not None:
            assert not np.array_equal(before, params)
        before = params
        w1, b1, w2, b2 = net.views(params)
        for j in range(N):
            x = torch.from_numpy(rng.standard_normal((M, d)).astype(np.float32)).to(dev()).to(BF)
            dy = torch.from_numpy((rng.standard_normal((M, d)) * 0.1).astype(np.float32)).to(dev()).to(BF)
            drop = Z.zero_dropout(0.2, 1000 + j, it)
            got = net.run(shards, x, dy, drop, grads[j])
            # each operator against its definition on the very inputs it was given
            ya, ea, za, eza = R.linear_forward(f64(x), w1.T, b1, act_name="gelu")
            check("a", got["a"], ya, ea)
            check("z", got["z"], za, eza)
            want, err, _, _ = R.linear_forward(f64(got["a"]), w2, b2, p=0.2, seed=1000 + j, offset=it, residual=f64(x))
            check("y", got["y"], want, err)
            check("d2", got["d2"], *R.dropout_grad(f64(dy), p=0.2, seed=1000 + j, offset=it))
            check("dz", got["dz"], *R.linear_grad_input(f64(got["d2"]), w2, act_name="gelu", z=f64(got["z"])))
            check("dx", got["dx"], *R.linear_grad_input(f64(got["dz"]), w1.T))
            g1, gb1, g2, gb2 = net.views(grads[j])
            want, err = R.linear_grad_weight(f64(got["dz"]), f64(x))
            check("g1", g1, want.T, err.T)
            check("gb1", gb1, *R.column_sums(f64(got["dz"])))
            check("g2", g2, *R.linear_grad_weight(f64(got["d2"]), f64(got["a"])))
            check("gb2", gb2, *R.column_sums(f64(got["d2"])))
            # what lies between the tensors stays as it was
            rest = torch.ones(N * net.S, dtype=torch.bool)
            for t in range(1, 5):
                rest[net.offsets[t]:net.offsets[t] + net.numels[t]] = False
            assert bool((grads[j].cpu()[rest] == 0).all())
        for r in range(N):
            slices = [g[r * net.S:(r + 1) * net.S].view(torch.int16) for g in grads]
            if it == 0:
                p = flat[r * net.S:(r + 1) * net.S].copy()
                m, v = np.zeros_like(p), np.zeros_like(p)
                slot = oracle.f32_to_bf16(p)
                oracle.step([to_host(s) for s in slices], p, m, v, slot, loss_scale=1.0, t=1, lr=1e-2, beta1=0.9,
                            beta2=0.999, eps=1e-8, wd=0.01)
            steps[r].step(slices)
            assert steps[r].state().t == it + 1
            if it == 0:
                assert np.array_equal(to_host(steps[r].current_slot()), slot)


def test_gradients_against_differences(Z):
    """Directional differences of sum(y * c) in 64 bits agree with the flat gradient: the
    whole chain of forward, dropout, activation and the three gradients."""
    d, inner, M = 72, 104, 64
    net = Mlp(Z, d, inner, 1)
    rng = np.random.default_rng(22)
    params = torch.from_numpy((rng.standard_normal(net.S) * 0.2).astype(np.float32)).to(dev()).to(BF)
    x = torch.from_numpy(rng.standard_normal((M, d)).astype(np.float32)).to(dev()).to(BF)
    c = torch.from_numpy(rng.standard_normal((M, d)).astype(np.float32)).to(dev()).to(BF)
    drop = Z.zero_dropout(0.3, 5, 6)
    grads = torch.zeros(net.S, dtype=F32, device=dev())
    got = net.run([params], x, c, drop, grads)
    p64, x64, c64 = f64(params), f64(x), f64(c)
    factor = R.drop_factor(M, d, 0.3, 5, 6)

    def loss(p, xx):
        w1, b1, w2, b2 = net.views(p)
        return float(((xx + (R.act("gelu", xx @ w1 + b1) @ w2.T + b2) * factor) * c64).sum())

    # bf16 activations and gradients between the operators: each of the four roundings
    # on the way is half a step, 2^-8 relative, of terms whose magnitudes add up to
    # less than the sums of absolute products below
    for k in range(4):
        v = rng.standard_normal(net.S) * (rng.random(net.S) < 0.3)
        h = 1e-5
        diff = (loss(p64 + h * v, x64) - loss(p64 - h * v, x64)) / (2 * h)
        have = float((f64(grads) * v).sum())
        scale = float(np.sqrt((f64(grads) ** 2 * v ** 2).sum()))
        # independent roundings of the terms: 4 * 2^-8 of their root sum of squares, five-fold
        assert abs(diff - have) <= 5 * 4 * 2.0 ** -8 * scale + 1e-6, (k, diff, have, scale)
    v = rng.standard_normal((M, d))
    h = 1e-5
    diff = (loss(p64, x64 + h * v) - loss(p64, x64 - h * v)) / (2 * h)
    # the residual's share of the gradient by x is c itself
    g = f64(got["dx"]) + c64
    have = float((g * v).sum())
    scale = float(np.sqrt((g ** 2 * v ** 2).sum()))
    assert abs(diff - have) <= 5 * 4 * 2.0 ** -8 * scale + 1e-6


def test_micro_batches_accumulate(Z):
    """Two micro-batches accumulated in f32 equal one of both."""
    d, inner, M = 64, 128, 96
    net = Mlp(Z, d, inner, 1)
    rng = np.random.default_rng(23)
    params = torch.from_numpy((rng.standard_normal(net.S) * 0.2).astype(np.float32)).to(dev()).to(BF)
    x = torch.from_numpy(rng.standard_normal((2 * M, d)).astype(np.float32)).to(dev()).to(BF)
    dy = torch.from_numpy(rng.standard_normal((2 * M, d)).astype(np.float32)).to(dev()).to(BF)
    one, two = (torch.zeros(net.S, dtype=F32, device=dev()) for _ in range(2))
    net.run([params], x, dy, None, one)
    net.run([params], x[:M], dy[:M], None, two)
    net.run([params], x[M:], dy[M:], None, two, accumulate=True)
    # the same bf16 operands in another grouping: fp32 sums of 192 terms
    err = R.sum_err(2 * M, 200.0)
    assert np.abs(f64(one) - f64(two)).max() <= 2 * err


def test_flat_linear_refuses(Z):
    with pytest.raises(Z.ZeroError):
        Z.FlatLinear([0, 64], [64, 8], 0, 1, 8, 9)
    with pytest.raises(Z.ZeroError):
        Z.FlatLinear([0, 64], [64, 7], 0, 1, 8, 8)
    layer = Z.FlatLinear([0, 64], [64, 8], 0, 1, 8, 8)
    x = torch.zeros((2, 8), dtype=BF, device=dev())
    with pytest.raises(Z.ZeroError):
        layer.forward(x)
    with pytest.raises(Z.ZeroError):
        layer.use(torch.zeros(70, dtype=BF, device=dev()))
    layer.use(torch.ones(72, dtype=BF, device=dev()))
    y, z = layer.forward(x)
    assert z is None and bool((y == 1).all())
    with pytest.raises(Z.ZeroError):
        layer.backward(x, x, torch.zeros(64, dtype=F32, device=dev()))


def test_bench_layer_mode(Z):
    """The layer mode of bench.py on a few tokens."""
    import json
    import os
    import subprocess
    import sys
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, os.path.join(root, "bench.py"), "--layer", "--config", "gpt2s", "--tokens", "130",
                        "--steps", "2", "--warmup", "1"], capture_output=True, text=True, timeout=110, cwd=root)
    assert r.returncode == 0, r.stderr
    line = json.loads(r.stdout.strip().splitlines()[-1])
    assert line["unit"] == "TFLOP/s" and line["value"] > 0 and line["config"]["tokens"] == 130
