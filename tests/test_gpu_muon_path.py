"""The norms and the matrix step as a training step uses them: a block whose tensors lie in
flat buffers, forward and backward against torch in 64 bits, and the step of its matrices,
whole and cut by shards, against the operators' own references."""
import numpy as np
import pytest
import torch

import muon_ref as R
from gpu_util import dev, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def flat_of(numels, align=8):
    offs, at = [], 0
    for n in numels:
        offs.append(at)
        at += -(-n // align) * align
    return offs, at


def test_a_block_forward_and_backward(Z):
    """h2 = h + W2 gelu(W1 norm(h) + b1) + b2, fetched out of two shards, back to the gradient
    buffer and to h. At most eight roundings to bf16 lie between the inputs and any of the
    results, each of 2^-8 of what it rounds: 2^-5 of a result's norm is allowed."""
    M, d, inner = 200, 96, 160
    g = torch.Generator(device=dev()).manual_seed(7)
    numels = [d, d, inner * d, inner, d * inner, d]
    offs, total = flat_of(numels)
    S = -(-total // 16) * 8
    params = torch.randn(2 * S, generator=g, device=dev()) * 0.2
    params[offs[0]:offs[0] + d] += 1
    params = params.to(BF)
    shards = [params[:S].contiguous(), params[S:].contiguous()]
    norm = Z.FlatNorm(offs, numels, 0, 1, d)
    up = Z.FlatLinear(offs, numels, 2, 3, d, inner, act=Z.ZERO_ACT_GELU)
    down = Z.FlatLinear(offs, numels, 4, 5, inner, d)
    h, dh2 = (torch.randn(M, d, generator=g, device=dev()).to(BF) for _ in range(2))
    a = torch.randn(M, d, generator=g, device=dev()).to(BF)         # what the block before adds to the stream
    for layer in (norm, up, down):
        layer.fetch(shards, S)
    say("block: forward, backward")
    y, s, stats = norm.forward(a, residual=h)
    x1, z = up.forward(y)
    h2, _ = down.forward(x1, residual=s)
    grads = torch.full((2 * S,), 3.0, dtype=F32, device=dev())
    before = grads.clone()
    dz = down.backward(dh2, x1, grads, below=(Z.ZERO_ACT_GELU, z, None))
    dy = up.backward(dz, y, grads)
    ds = norm.backward(dy, s, stats, grads, residual_grad=dh2)
    # the same in 64 bits
    P = params.cpu().double()
    leaf = [P[o:o + n].clone().requires_grad_() for o, n in zip(offs, numels)]
    s64 = (a.cpu().double() + h.cpu().double()).requires_grad_()
    y64 = torch.nn.functional.layer_norm(s64, (d,), leaf[0], leaf[1], 1e-5)
    x64 = torch.nn.functional.gelu(y64 @ leaf[2].view(inner, d).T + leaf[3], approximate="tanh")
    want = s64 + x64 @ leaf[4].view(d, inner).T + leaf[5]
    want.backward(dh2.cpu().double())

    def near(name, got, ref):
        got, ref = got.cpu().double().reshape(-1), ref.detach().reshape(-1)
        assert float((got - ref).norm()) <= 2.0 ** -5 * float(ref.norm()), name

    near("h2", h2, want)
    near("ds", ds, s64.grad)
    covered = torch.zeros(2 * S, dtype=torch.bool, device=dev())
    for k, (o, n) in enumerate(zip(offs, numels)):
        near(f"gradient {k}", grads[o:o + n], leaf[k].grad)
        covered[o:o + n] = True
    assert torch.equal(grads[~covered], before[~covered])
    # accumulated: what the norm adds to what is there
    twice = grads.clone()
    norm.backward(dy, s, stats, twice, residual_grad=dh2, accumulate=True)
    for k in (0, 1):
        near(f"twice {k}", twice[offs[k]:offs[k] + d], 2 * leaf[k].grad)
    norm.release()
    with pytest.raises(Z.ZeroError, match="fetch or use first"):
        norm.forward(a)


def replicas_of(rng, n, N, dtype, scale):
    return [torch.from_numpy((rng.standard_normal(n) * 1e-2 * scale).astype(np.float32)).to(dev()).to(dtype)
            for _ in range(N)]


def averaged(reps, loss_scale):
    acc = reps[0].float().cpu().numpy()
    for r in reps[1:]:
        acc = acc + r.float().cpu().numpy()
    return acc * np.float32(1.0 / (len(reps) * loss_scale))


MATRICES = [(0, 24, 40), (960, 24, 40), (1920, 24, 40), (2880, 70, 33), (5200, 8, 200), (6800, 24, 40)]


def test_step_of_whole_matrices(Z):
    """Three steps against the operators' references: gradient, momentum and update bit for bit,
    the orthogonal forms within their bounds; one of them overflows and leaves everything."""
    S, N, scale = 7768, 3, 1024.0
    rng = np.random.default_rng(3)
    p0 = torch.from_numpy(rng.standard_normal(S).astype(np.float32)).to(dev())
    step = Z.MuonShardStep(S, N, Z.ZERO_BF16, p0, MATRICES, lr=0.02, weight_decay=0.1, loss_scale=scale, dynamic=True)
    assert sorted(u.shape[0] for u, _, _ in step.stacks) == [1, 1, 1, 3]
    p, m = p0.cpu().numpy(), np.zeros(S, np.float32)
    for k in range(3):
        reps = replicas_of(rng, S, N, BF, scale)
        if k == 1:
            reps[2][77] = float("inf")
        say("matrix step", k)
        st, verdict = step.step(reps)
        if k == 1:
            assert verdict == Z.ZERO_SKIP and st.overflow == 1 and step.loss_scale == scale / 2
            scale /= 2
        else:
            assert verdict == Z.ZERO_COMMIT and st.overflow == 0
            m, u = R.momentum(averaged(reps, scale), m, 0.95, True)
            u = torch.from_numpy(u).to(BF)
            assert torch.equal(step.u.cpu(), u)
            o = step.o.cpu()
            rest = torch.ones(S, dtype=torch.bool)
            for at, r, c in MATRICES:
                want, each, whole = R.bounds(u[at:at + r * c].double().numpy().reshape(r, c),
                                             scale=0.2 * np.sqrt(max(r, c)))
                d = np.abs(o[at:at + r * c].double().numpy().reshape(r, c) - want)
                assert (d <= each).all() and np.linalg.norm(d) <= whole
                rest[at:at + r * c] = False
            assert bool((o[rest] == 0).all())
            p = R.update(p, o.float().numpy(), 0.02, 0.1)
        assert np.array_equal(step.m.cpu().numpy(), m) and np.array_equal(step.master.cpu().numpy(), p)
        assert torch.equal(step.slot.view(BF).cpu(), torch.from_numpy(p).to(BF))
    assert step.t == 2
    # resumed, the next step goes on as it would have
    again = Z.MuonShardStep(S, N, Z.ZERO_BF16, p0, MATRICES, lr=0.02, weight_decay=0.1)
    again.load_state_dict(step.state_dict())
    reps = replicas_of(rng, S, N, BF, scale)
    step.step(reps)
    again.step(reps)
    assert torch.equal(step.master, again.master) and torch.equal(step.slot, again.slot) and step.t == again.t == 3


def test_step_of_cut_matrices(Z):
    """Two shards that cut a matrix, with an exchange of u between them: as one shard of both.
    Where one overflows and they agree, neither writes anything."""
    S, N = 3884, 2
    rng = np.random.default_rng(4)
    p0 = torch.from_numpy(rng.standard_normal(2 * S).astype(np.float32)).to(dev())
    kw = dict(lr=0.01, weight_decay=0.05)
    one = Z.MuonShardStep(2 * S, N, Z.ZERO_F32, p0, MATRICES, **kw)
    two = [Z.MuonShardStep(S, N, Z.ZERO_F32, p0[r * S:(r + 1) * S].clone(), MATRICES, shard_off=r * S, **kw)
           for r in range(2)]
    assert one.whole and not two[0].whole
    reps = replicas_of(rng, 2 * S, N, F32, 1.0)
    parts = [[r[k * S:(k + 1) * S].clone() for r in reps] for k in range(2)]
    with pytest.raises(Z.ZeroError, match="exchange"):
        two[0].step(parts[0])
    say("cut matrices")
    one.step(reps)
    for s, mine in zip(two, parts):
        s.reduce(mine)
        s.momentum()
    whole = torch.cat([s.u_shard for s in two])
    for s in two:
        s.u.copy_(whole[s.u_off:s.u_off + s.u.numel()])
        s.update()
    for k, s in enumerate(two):
        assert s.commit(s.read_stats()) == Z.ZERO_COMMIT
        assert torch.equal(s.m, one.m[k * S:(k + 1) * S])
        # a matrix's orthogonal form within twice its bound, the update itself bit for bit
        want = R.update(p0[k * S:(k + 1) * S].cpu().numpy(), s.o_shard.float().cpu().numpy(), 0.01, 0.05)
        assert np.array_equal(s.master.cpu().numpy(), want)
        # orthogonal forms of the same matrices, by other batches
        off = (s.o_shard.double() - one.o_shard[k * S:(k + 1) * S].double()).norm()
        assert float(off) <= 2 * (2e-3 + 2.0 ** -9) * float(one.o_shard.double().norm())
    held = [(s.p.clone(), s.m.clone(), s.slot.clone()) for s in two]
    parts[1][0][5] = float("nan")

    def agree(stats):
        stats.copy_(two[1].stats)

    for s, mine in zip(reversed(two), reversed(parts)):
        st, verdict = s.step(mine, agree=agree, exchange=lambda u: None)
        assert verdict == Z.ZERO_SKIP and st.overflow == 1
    for s, was in zip(two, held):
        assert all(torch.equal(a, b) for a, b in zip((s.p, s.m, s.slot), was)) and s.t == 1


def test_a_step_on_another_stream_and_captured(Z):
    """The three parts on a stream of their own, and in a graph that is replayed on new
    gradients between the program's own work, against the same steps run eagerly."""
    S, N = 7768, 2
    rng = np.random.default_rng(5)
    p0 = torch.from_numpy(rng.standard_normal(S).astype(np.float32)).to(dev())

    def new():
        return Z.MuonShardStep(S, N, Z.ZERO_F32, p0, MATRICES, lr=0.02)

    sets = [replicas_of(rng, S, N, F32, 1.0) for _ in range(3)]
    eager = new()
    for reps in sets:
        eager.step(reps)
    s = torch.cuda.Stream()
    other = new()
    torch.cuda.synchronize()
    for reps in sets:
        st, verdict = other.step(reps, stream=s)
        assert verdict == Z.ZERO_COMMIT
    torch.cuda.synchronize()
    assert torch.equal(other.master, eager.master)
    held, fixed = new(), [torch.zeros(S, device=dev()) for _ in range(N)]
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        held.reduce(fixed)
        held.momentum()
        held.update()
    for reps in sets:
        for a, b in zip(fixed, reps):
            a.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
    assert torch.equal(held.master, eager.master) and torch.equal(held.m, eager.m)


def test_refuses(Z):
    p0 = torch.zeros(100, device=dev())
    with pytest.raises(Z.ZeroError, match="overlap"):
        Z.MuonShardStep(100, 1, Z.ZERO_F32, p0, [(0, 5, 10), (49, 5, 10)], lr=0.1)
    with pytest.raises(Z.ZeroError, match="matrix at -1"):
        Z.MuonShardStep(100, 1, Z.ZERO_F32, p0, [(-1, 5, 10)], lr=0.1)
    step = Z.MuonShardStep(100, 1, Z.ZERO_F32, p0, [(0, 5, 10)], lr=0.1)
    with pytest.raises(Z.ZeroError, match="replicas"):
        step.step([p0, p0])
    for bad in (p0[:99], p0.bfloat16(), p0.cpu(), torch.zeros(200, device=dev())[::2]):
        with pytest.raises(Z.ZeroError, match="a replica of"):
            step.step([bad])
    assert step.t == 0
