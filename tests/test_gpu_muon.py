"""GPU tests of the matrix step's operators against tests/muon_ref.py."""
import zlib

import numpy as np
import pytest
import torch

import muon_ref as R
from gpu_util import dev, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TY = {"bf16": BF, "f32": F32}
SENT = -12345.0


def rng_of(*case):
    return np.random.default_rng(zlib.crc32(repr(case).encode()))


class Stack:
    """Matrices inside a larger buffer: rows longer than their columns, matrices further
    apart than their rows, a base at any element."""

    def __init__(self, batch, rows, cols, dtype, *, pad=0, gap=0, shift=0, fill=None, around=SENT):
        ld = cols + pad
        stride = rows * ld + gap
        self.raw = torch.full((64 + shift + batch * stride + 64,), around, dtype=dtype, device=dev())
        self.t = self.raw.as_strided((batch, rows, cols), (stride, ld, 1), 64 + shift)
        if fill is not None:
            self.t.copy_(torch.from_numpy(fill))
        self.before = self.raw.clone()

    def intact_outside(self):
        inside = torch.zeros_like(self.raw, dtype=torch.bool)
        inside.as_strided(self.t.shape, self.t.stride(), self.t.storage_offset()).fill_(True)
        same = (self.raw == self.before) | (self.raw.isnan() & self.before.isnan())
        return bool((same | inside).all())


def falling(rng, *shape):
    """Matrices of a few strong directions that fall off over noise, as momenta are."""
    B, r, c = shape
    k = min(r, c, 12)
    x = (rng.standard_normal((B, r, k)) * np.exp(-np.arange(k) / 3)) @ rng.standard_normal((B, k, c))
    return (1e-3 * (x + 0.1 * rng.standard_normal(shape))).astype(np.float32)


def check(o, x, **kw):
    """Each matrix of o against the formula for that of x (tensors)."""
    o, x = o.cpu().double().numpy(), x.cpu().double().numpy()
    for k in range(o.shape[0]):
        want, each, whole = R.bounds(x[k], **kw)
        d = np.abs(o[k] - want)
        bad = ~(d <= each)
        assert not bad.any(), (k, int(bad.sum()), np.argwhere(bad)[0], float(d.max()), float(np.min(each)))
        assert np.linalg.norm(d) <= whole, (k, float(np.linalg.norm(d)), whole)


# single elements, rows and columns; edges of 8, of the 128 and 256 tiles and of the padding;
# wide, tall and square; stacks
SIZES = [(1, 1, 1), (1, 1, 300), (1, 300, 1), (3, 2, 3), (2, 7, 9), (1, 8, 8), (2, 64, 64), (1, 65, 127), (2, 127, 65),
         (1, 128, 128), (1, 129, 128), (1, 128, 129), (5, 100, 260), (2, 256, 256), (1, 257, 255), (1, 300, 700),
         (1, 700, 300), (1, 33, 2000), (1, 2000, 33), (1, 513, 512), (4, 384, 640), (1, 768, 768), (1, 1001, 530)]


@pytest.mark.parametrize("ty", ["bf16", "f32"])
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_sizes(Z, size, ty):
    B, r, c = size
    rng = rng_of(1, size, ty)
    pad, gap, shift = [(0, 0, 0), (8, 16, 0), (1, 3, 1), (5, 0, 3)][(B + r + c) % 4]
    x = Stack(B, r, c, TY[ty], pad=pad, gap=gap, shift=shift, fill=falling(rng, B, r, c), around=float("nan"))
    o = Stack(B, r, c, BF, pad=pad, gap=gap, shift=shift)
    say("orthogonalize", size, ty, pad, gap, shift)
    assert Z.zero_orthogonalize(x.t, out=o.t) is o.t
    check(o.t, x.t)
    assert o.intact_outside() and x.intact_outside()


@pytest.mark.parametrize("size", [(96, 200), (200, 96), (150, 150)], ids=str)
@pytest.mark.parametrize("kind", ["normal", "rank1", "rank6", "fall"])
def test_spectra(Z, kind, size):
    """Whatever the fall of the singular values."""
    r, c = size
    rng = rng_of(2, kind, size)
    if kind == "normal":
        x = rng.standard_normal(size)
    elif kind == "fall":
        k = min(size)
        q = [np.linalg.qr(rng.standard_normal((n, k)))[0] for n in size]
        x = (q[0] * np.logspace(0, -5, k)) @ q[1].T
    else:
        k = int(kind[4:])
        x = rng.standard_normal((r, k)) @ rng.standard_normal((k, c))
    x = torch.from_numpy(x.astype(np.float32)).to(dev())[None]
    say("orthogonalize", kind, size)
    check(Z.zero_orthogonalize(x), x)


@pytest.mark.parametrize("kw", [dict(steps=1), dict(steps=2, scale=-3.5), dict(steps=8, coefficients=(1.5, -0.5, 0.0)),
                                dict(steps=3, coefficients=[(3.4, -4.7, 2.0), (2.0, -1.5, 0.5), (1.875, -1.25, 0.375)]),
                                dict(eps=1e-2), dict(scale=0.2 * 20.0), dict(steps=12, coefficients=(2.0, -1.5, 0.5))],
                         ids=str)
def test_parameters(Z, kw):
    rng = rng_of(3, str(kw))
    for shape in ((2, 60, 140), (1, 140, 60)):
        x = torch.from_numpy(falling(rng, *shape)).to(dev())
        say("orthogonalize", kw, shape)
        check(Z.zero_orthogonalize(x, **kw), x, **kw)


def apart(a, b):
    """The norm of a - b over that of b, matrix by matrix. Two results for the same matrix are
    each within 2e-3 and o's rounding (2^-9) of the formula's."""
    a, b = a.double(), b.double()
    return float(((a - b).square().sum((-2, -1)) / b.square().sum((-2, -1))).sqrt().max())


BOTH = 2 * (2e-3 + 2.0 ** -9)


def test_a_matrix_alone_in_a_stack_and_transposed(Z):
    """The same call gives the same bits; a stack and its matrices alone, whose sums may be
    split in other ways, the same within twice the bound; a 2-D tensor is a stack of one."""
    rng = rng_of(4)
    x = torch.from_numpy(falling(rng, 7, 200, 330)).to(dev()).to(BF)
    o = Z.zero_orthogonalize(x)
    assert torch.equal(o, Z.zero_orthogonalize(x))
    for k in range(7):
        one = Z.zero_orthogonalize(x[k])
        check(one[None], x[k][None])
        assert torch.equal(one, Z.zero_orthogonalize(x[k:k + 1])[0])
        assert apart(one, o[k]) <= BOTH
    check(Z.zero_orthogonalize(x[::2]), x[::2])
    t = Z.zero_orthogonalize(x.transpose(1, 2).contiguous())
    check(t.transpose(1, 2), x)


def test_scale_of_x_does_not_matter(Z):
    """Powers of two change nothing, far beyond where a sum of squares would leave fp32."""
    x = torch.from_numpy(falling(rng_of(5), 1, 90, 150)).to(dev())
    o = Z.zero_orthogonalize(x, eps=1e-30)
    for e in (-60, -20, 40, 120):
        assert torch.equal(Z.zero_orthogonalize(x * 2.0 ** e, eps=1e-30), o), e


def test_zeros_infinities_and_nan(Z):
    """Zeros give zeros; what is not finite stays in its matrix."""
    x = torch.from_numpy(falling(rng_of(6), 5, 140, 270)).to(dev())
    clean = Z.zero_orthogonalize(x)
    x[1] = 0.0
    x[2, 139, 269] = float("inf")
    x[3, 0, 0] = float("nan")
    o = Z.zero_orthogonalize(x)
    assert bool((o[1] == 0).all()) and bool(o[2].isnan().all()) and bool(o[3].isnan().all())
    assert torch.equal(o[[0, 4]], clean[[0, 4]])


def test_empty(Z):
    for shape in ((0, 4, 8), (3, 0, 8), (3, 4, 0), (0, 5), (5, 0)):
        x = torch.empty(shape, dtype=BF, device=dev())
        assert Z.zero_orthogonalize(x).shape == x.shape


# by the products' tiles: 64 wide, 128 in each of their two kinds, 256 whole, split, and whole
# and split together, of wide and tall matrices
@pytest.mark.parametrize("size", [(1, 4096, 1000), (2, 1100, 2304), (1, 640, 11008), (30, 256, 512), (40, 700, 500),
                                  (1, 4096, 4096), (1, 2500, 9000), (1, 9000, 2500), (4, 2304, 4096), (3, 5000, 2304), (4, 4096, 4096), (4, 4096, 2304)],
                         ids=str)
def test_large(Z, size):
    """Sizes of many tiles, where the fp64 formula runs on the device: the norm of the error is
    within the documented 2e-3 and o's rounding (2^-9 in the mean square of a bf16 rounding)."""
    B, r, c = size
    x = torch.from_numpy(falling(rng_of(7, size), B, r, c)).to(dev())
    say("orthogonalize", size)
    o = Z.zero_orthogonalize(x).double()
    X = x.double()
    X = X / X.square().sum((1, 2), keepdim=True).sqrt()
    tall = r > c
    X = X.transpose(1, 2).contiguous() if tall else X
    for _ in range(5):
        A = torch.bmm(X, X.transpose(1, 2).contiguous())
        X = R.COEF[0] * X + torch.bmm(R.COEF[1] * A + R.COEF[2] * torch.bmm(A, A), X)
    X = X.transpose(1, 2) if tall else X
    rel = (o - X).square().sum((1, 2)).sqrt() / X.square().sum((1, 2)).sqrt()
    assert float(rel.max()) <= 2e-3 + 2.0 ** -9, rel.max()
    big = X.square().mean((1, 2), keepdim=True).sqrt()
    assert float(((o - X).abs() - 2.0 ** -8 * X.abs()).div(big).max()) < 0.05      # 25 standard deviations of 2e-3


def test_groups(Z):
    """A stack whose intermediate results pass 4 GiB goes in groups."""
    B, r, c = 180, 1024, 4096
    need = Z.zero_orthogonalize_workspace_bytes(B, r, c)
    assert need <= 4 << 30 and need < B * Z.zero_orthogonalize_workspace_bytes(1, r, c)
    g = torch.Generator(device=dev()).manual_seed(11)
    x = torch.empty(B, r, c, dtype=BF, device=dev()).normal_(generator=g)
    o = Z.zero_orthogonalize(x)
    n = need // Z.zero_orthogonalize_workspace_bytes(1, r, c)
    for k in (0, n - 1, n, B - 1):
        assert apart(Z.zero_orthogonalize(x[k]), o[k]) <= BOTH, k


def test_streams_and_graphs(Z):
    """Two calls at once with workspaces of their own, and a captured one replayed on new
    inputs between the program's own work."""
    rng = rng_of(8)
    xs = [torch.from_numpy(falling(rng, 2, 300, 500)).to(dev()).to(BF) for _ in range(2)]
    want = [Z.zero_orthogonalize(x) for x in xs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [Z.zero_orthogonalize(x, stream=s) for x, s in zip(xs, streams)]
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    x = xs[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o = Z.zero_orthogonalize(x)
    for k in (1, 0, 1):
        x.copy_(xs[k])
        o.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(o, want[k])


@pytest.mark.parametrize("n", [1, 7, 8, 9, 2048, 2049, 100003])
@pytest.mark.parametrize("nesterov", [True, False])
def test_momentum_bits(Z, n, nesterov):
    """Every product and sum one fp32 operation, at any base address; nothing outside written."""
    rng = rng_of(21, n, nesterov)
    for grad, out, shift in (("f32", "bf16", 0), ("bf16", "f32", 1), ("f32", "f32", 3), ("bf16", "bf16", 5)):
        g, m = (Stack(1, 1, n, ty, shift=shift, fill=rng.standard_normal((1, 1, n)).astype(np.float32))
                for ty in (TY[grad], F32))
        u = Stack(1, 1, n, TY[out], shift=shift)
        m2, u2 = R.momentum(g.t[0, 0].float().cpu().numpy(), m.t[0, 0].cpu().numpy(), 0.95, nesterov)
        Z.zero_muon_momentum(g.t[0, 0], m.t[0, 0], mu=0.95, nesterov=nesterov, u=u.t[0, 0])
        assert np.array_equal(m.t[0, 0].cpu().numpy(), m2)
        assert torch.equal(u.t[0, 0].cpu(), torch.from_numpy(u2).to(TY[out]))
        assert g.intact_outside() and m.intact_outside() and u.intact_outside()
    # u over grad
    g, m = (torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(dev()) for _ in range(2))
    m2, u2 = R.momentum(g.cpu().numpy(), m.cpu().numpy(), 0.9, nesterov)
    Z.zero_muon_momentum(g, m, mu=0.9, nesterov=nesterov, u=g)
    assert np.array_equal(g.cpu().numpy(), u2) and np.array_equal(m.cpu().numpy(), m2)


@pytest.mark.parametrize("n", [1, 7, 8, 9, 2048, 2049, 100003])
def test_update_bits(Z, n):
    rng = rng_of(22, n)
    for shift, decay, with_slot in ((0, 0.1, True), (3, 0.0, True), (1, 0.5, False)):
        p, o = (Stack(1, 1, n, ty, shift=shift, fill=rng.standard_normal((1, 1, n)).astype(np.float32))
                for ty in (F32, BF))
        slot = Stack(1, 1, n, BF, shift=shift)
        want = R.update(p.t[0, 0].cpu().numpy(), o.t[0, 0].float().cpu().numpy(), 0.02, decay)
        Z.zero_muon_update(p.t[0, 0], o.t[0, 0], lr=0.02, weight_decay=decay, slot=slot.t[0, 0] if with_slot else None)
        assert np.array_equal(p.t[0, 0].cpu().numpy(), want)
        if with_slot:
            assert torch.equal(slot.t[0, 0].cpu(), torch.from_numpy(want).to(BF))
        assert p.intact_outside() and o.intact_outside() and slot.intact_outside()


def test_overflow_leaves_everything(Z):
    n = 5000
    rng = rng_of(23)
    g, m, p = (torch.from_numpy(rng.standard_normal(n).astype(np.float32)).to(dev()) for _ in range(3))
    u, slot = torch.full((n,), 7.0, dtype=BF, device=dev()), torch.full((n,), 9, dtype=torch.int16, device=dev())
    for flag in (1, 0):
        stats = torch.tensor([flag, 0, 0, 0], dtype=torch.int32, device=dev())
        m0, p0 = m.clone(), p.clone()
        Z.zero_muon_momentum(g, m, u=u, stats=stats)
        Z.zero_muon_update(p, u, lr=0.1, slot=slot, stats=stats)
        assert torch.equal(m, m0) == bool(flag) and torch.equal(p, p0) == bool(flag)
        assert bool((u == 7).all()) == bool(flag) and bool((slot == 9).all()) == bool(flag)


def test_refuses(Z):
    x = torch.zeros(4, 8, dtype=BF, device=dev())
    f = Z.zero_orthogonalize
    for call, word in ((lambda: f(x.half()), "neither"), (lambda: f(x[0]), "neither a matrix"),
                       (lambda: f(x.t()), "stride"), (lambda: f(x, out=x[:2]), "out has shape"),
                       (lambda: f(x, out=x.float()), "out is"), (lambda: f(x, out=x), "overlap"),
                       (lambda: f(x[None].expand(3, 4, 8)), "batch stride"),
                       (lambda: f(x, steps=0), "steps"), (lambda: f(x, eps=0.0), "eps"),
                       (lambda: f(x, coefficients=(1.0, 2.0)), "coefficients"),
                       (lambda: f(x, workspace=torch.zeros(4, device=dev())), "ws_bytes"),
                       (lambda: Z.zero_muon_momentum(x[0], x[0]), "momentum"),
                       (lambda: Z.zero_muon_momentum(x[0], torch.zeros(9, device=dev())), "momentum"),
                       (lambda: Z.zero_muon_momentum(x[:, 0], torch.zeros(4, device=dev())), "grad"),
                       (lambda: Z.zero_muon_momentum(x[0], torch.zeros(8, device=dev()), stats=x[0, :2]), "stats"),
                       (lambda: Z.zero_muon_update(x[0], x[0], lr=0.1), "p is"),
                       (lambda: Z.zero_muon_update(torch.zeros(8, device=dev()), x[0], lr=-0.1), "lr")):
        say("refused for", word)
        with pytest.raises(Z.ZeroError, match=word):
            call()
