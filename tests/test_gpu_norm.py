"""GPU tests of the norms and their gradient against tests/norm_ref.py in 64 bits. Every
matrix of a case lies in a larger buffer: rows longer than their columns, a base at any
element, NaN in what inputs leave unused and a sentinel in what outputs must not touch.
"""
import zlib

import numpy as np
import pytest
import torch

import norm_ref as R
from gpu_util import dev, say
from test_gpu_layer import BF, F32, TY, Mat, close, inp, rand

pytestmark = pytest.mark.gpu


def rng_of(*case):
    return np.random.default_rng(zlib.crc32(repr(case).encode()))


def vec(rng, N, mean=0.0, dtype=BF):
    return torch.from_numpy(mean + 0.3 * rand(rng, N)).to(dev()).to(dtype)


def v64(t, N, fill):
    return np.full(N, fill) if t is None else t.cpu().double().numpy()


KINDS = ["layer", "rms"]
# edges of 8, of a wave's 512 columns, and of each kernel's reach (512, 1024, 2048, 4096, 8192, 16384)
SIZES = [(1, 1), (1, 768), (3, 7), (5, 8), (4, 9), (2, 511), (9, 512), (7, 513), (130, 768), (33, 1001), (17, 1024),
         (6, 1025), (11, 2048), (5, 2049), (9, 4096), (3, 4100), (4, 8191), (2, 8200), (3, 11008), (2, 16384),
         (2, 16385), (3, 20011), (1029, 64), (700, 40)]
PLACES = [(0, 0), (8, 0), (1, 0), (0, 1), (5, 3)]
TYPES = [(a, b, c) for a in ("bf16", "f32") for b in ("bf16", "f32") for c in ("bf16", "f32")]


def forward_case(Z, rng, M, N, kind, types, *, residual=False, weight=True, bias=True, place=(0, 0), eps=1e-5,
                 mean=0.5, scale=1.0, kwargs=None):
    tx, ts, ty = types
    pad, shift = place

    def rows(ty):
        m = Mat(M, N, TY[ty], ld=N + pad, shift=shift, fill=(mean + rand(rng, M, N)) * np.float32(scale),
                pad=float("nan"))
        return m

    def out(ty):
        return Mat(M, N, TY[ty], ld=N + pad, shift=shift)

    x, res = rows(tx), rows(ts) if residual else None
    w, b = vec(rng, N, 1.0) if weight else None, vec(rng, N) if bias else None
    y, s = out(ty), out(ts) if residual else None
    st = Mat(M, 2, F32)
    k = Z.ZERO_NORM_LAYER if kind == "layer" else Z.ZERO_NORM_RMS
    got = Z.zero_norm_forward(x.t, w, b, kind=k, eps=eps, residual=res.t if residual else None,
                              sum=s.t if residual else None, y=y.t, stats=st.t, **(kwargs or {}))
    assert got[0] is y.t and got[-1] is st.t and len(got) == (3 if residual else 2)
    s64 = x.f64()
    if residual:
        want = x.f64() + res.f64()
        close("sum", s.t, want, (R.U[ts] * (1 + R.u) + R.u) * np.abs(want) + 2.0 ** -149)
        s64 = s.f64()                   # what is stored is what is normed
        assert s.intact_outside()
    want, err, stats, es = R.forward(s64, v64(w, N, 1.0), v64(b, N, 0.0), rms=kind == "rms", eps=eps, out=ty)
    close("stats", st.t, stats, es + 2.0 ** -140)
    close("y", y.t, want, err)
    assert y.intact_outside() and st.intact_outside()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward_sizes(Z, size, kind):
    M, N = size
    place, types = PLACES[(M + N) % 5], TYPES[(3 * M + N + (kind == "rms")) % 8]
    say("norm forward", size, kind, types, place)
    for residual in (False, True):
        forward_case(Z, rng_of(1, size, kind, residual), M, N, kind, types, residual=residual, place=place)


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("kind", KINDS)
def test_forward_types(Z, types, kind):
    for N in (200, 1500, 3000):
        say("norm forward", types, kind, N)
        forward_case(Z, rng_of(2, types, kind, N), 13, N, kind, types, residual=True, place=(3, 1))
        forward_case(Z, rng_of(3, types, kind, N), 13, N, kind, types)


@pytest.mark.parametrize("kind", KINDS)
def test_forward_without_weight_or_bias(Z, kind):
    for weight, bias in ((False, False), (True, False), (False, True)):
        say("norm forward", kind, weight, bias)
        forward_case(Z, rng_of(4, kind, weight, bias), 9, 300, kind, ("f32", "f32", "f32"), weight=weight, bias=bias)


@pytest.mark.parametrize("mean,scale,eps", [(1000.0, 1.0, 1e-5), (0.0, 1e-12, 1e-5), (0.0, 1e-12, 0.0), (0.0, 1e15, 0.0),
                                            (0.0, 1.0, 10.0)])
def test_forward_values(Z, mean, scale, eps):
    """A mean that is large beside the differences; tiny and huge rows; eps of all sizes."""
    for kind in KINDS:
        say("norm forward", kind, mean, scale, eps)
        forward_case(Z, rng_of(5, kind, mean, scale, eps), 6, 769, kind, ("f32", "f32", "f32"), mean=mean, scale=scale,
                     eps=eps)


@pytest.mark.parametrize("N", [40, 900, 3000, 17000])
def test_infinities_nan_and_constant_rows(Z, N):
    """They stay in their rows; a constant row gives the bias, and NaN only with eps 0."""
    rng = rng_of(6, N)
    x = torch.from_numpy(rand(rng, 6, N)).to(dev())
    clean = Z.zero_norm_forward(x, dtype=F32)
    x[1, N // 2], x[2, 3], x[3] = float("inf"), float("nan"), 0.0
    b = vec(rng, N)
    y = Z.zero_norm_forward(x, None, None, dtype=F32)
    assert torch.equal(y[[0, 4, 5]], clean[[0, 4, 5]])
    assert bool(y[1:3].isnan().all()) and bool((y[3] == 0).all())
    assert torch.equal(Z.zero_norm_forward(x, None, b, dtype=F32)[3], b.float())
    assert bool(Z.zero_norm_forward(x, eps=0.0, dtype=F32)[3].isnan().all())


@pytest.mark.parametrize("N", [100, 1024, 5000, 20000])
def test_forward_in_place(Z, N):
    """y over x or the residual, sum over the other: as from separate buffers."""
    rng = rng_of(7, N)
    x, r = (torch.from_numpy(rand(rng, 21, N)).to(dev()).to(BF) for _ in range(2))
    w = vec(rng, N, 1.0)
    y, s, st = Z.zero_norm_forward(x, w, residual=r, stats=True)
    for y_over in (True, False):
        a, b = x.clone(), r.clone()
        got = Z.zero_norm_forward(a, w, residual=b, y=a if y_over else b, sum=b if y_over else a, stats=True)
        assert all(torch.equal(p, q) for p, q in zip(got, (y, s, st)))
    a = x.clone()
    assert torch.equal(Z.zero_norm_forward(a, w, y=a), Z.zero_norm_forward(x, w))
    # a residual gives what an addition and a call without one give
    assert torch.equal(y, Z.zero_norm_forward(s, w))


def grad_case(Z, rng, M, N, kind, types, *, grad="f32", residual=False, weight=True, sums=(True, True),
              accumulate=False, place=(0, 0)):
    td, tx, to = types
    pad, shift = place

    def rows(ty, scale=1.0):
        return Mat(M, N, TY[ty], ld=N + pad, shift=shift, fill=rand(rng, M, N, scale=scale) + np.float32(0.1),
                   pad=float("nan"))

    dy, x, res = rows(td), rows(tx), rows(to) if residual else None
    w = vec(rng, N, 1.0) if weight else None
    x64 = x.f64()
    mean = x64.mean(1) if kind == "layer" else np.zeros(M)
    rstd = ((x64 - mean[:, None]) ** 2).mean(1) + 1e-5
    stats = torch.from_numpy(np.stack((mean, rstd ** -0.5), 1).astype(np.float32)).to(dev())
    dx = Mat(M, N, TY[to], ld=N + pad, shift=shift)
    dw, db = (Mat(1, N, TY[grad], shift=shift, fill=rand(rng, 1, N)) if s else None for s in sums)
    old = [m.f64()[0] if m is not None and accumulate else None for m in (dw, db)]
    k = Z.ZERO_NORM_LAYER if kind == "layer" else Z.ZERO_NORM_RMS
    got = Z.zero_norm_grad(dy.t, x.t, w, stats, kind=k, residual_grad=res.t if residual else None, dx=dx.t,
                           dweight=None if dw is None else dw.t[0], dbias=None if db is None else db.t[0],
                           accumulate=accumulate)
    assert got is dx.t
    wants = R.grad(dy.f64(), x64, v64(w, N, 1.0), stats.cpu().double().numpy(), rms=kind == "rms",
                   res=res.f64() if residual else None, out=to, old_w=old[0], old_b=old[1], grad_out=grad)
    close("dx", dx.t, *wants[0])
    assert dx.intact_outside()
    for name, m, (want, err) in (("dw", dw, wants[1]), ("db", db, wants[2])):
        if m is not None:
            close(name, m.t[0], want, err)
            assert m.intact_outside()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("size", SIZES + [(0, 40), (0, 9000), (5000, 24), (600, 1030)], ids=str)
def test_grad_sizes(Z, size, kind):
    M, N = size
    types, place = TYPES[(M + 3 * N + (kind == "rms")) % 8], PLACES[(M + 2 * N) % 5]
    say("norm grad", size, kind, types, place)
    for residual in (False, True):
        grad_case(Z, rng_of(11, size, kind, residual), M, N, kind, types, residual=residual, accumulate=residual,
                  grad=("f32", "bf16")[(M + N) % 2], place=place)


@pytest.mark.parametrize("types", TYPES, ids=str)
@pytest.mark.parametrize("kind", KINDS)
def test_grad_types(Z, types, kind):
    for N, grad in ((200, "bf16"), (1500, "f32"), (5000, "bf16"), (17000, "f32")):
        say("norm grad", types, kind, N, grad)
        grad_case(Z, rng_of(12, types, kind, N), 13, N, kind, types, grad=grad, residual=True, place=(3, 1))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("sums", [(True, False), (False, True), (False, False)], ids=str)
def test_grad_of_some(Z, kind, sums):
    for N in (300, 3000, 17000):
        say("norm grad", kind, sums, N)
        grad_case(Z, rng_of(13, kind, sums, N), 40, N, kind, ("bf16", "bf16", "bf16"), sums=sums, weight=sums[1])


@pytest.mark.parametrize("N", [100, 1024, 5000, 20000])
def test_grad_in_place(Z, N):
    """dx over dy, x or the residual's gradient: as from separate buffers."""
    rng = rng_of(14, N)
    dy, x, r = (torch.from_numpy(rand(rng, 21, N)).to(dev()).to(BF) for _ in range(3))
    st = Z.zero_norm_forward(x, stats=True)[1]

    def run(dy, x, r, dx):
        dw, db = torch.empty(N, device=dev()), torch.empty(N, device=dev())
        return Z.zero_norm_grad(dy, x, None, st, residual_grad=r, dx=dx, dweight=dw, dbias=db), dw, db

    want = run(dy, x, r, None)
    for k in range(3):
        a = [dy.clone(), x.clone(), r.clone()]
        assert all(torch.equal(p, q) for p, q in zip(run(*a, a[k]), want))


@pytest.mark.parametrize("kind", KINDS)
def test_gradient_is_that_of_the_forward_pass(Z, kind):
    """dx, dw and db against differences of the library's own forward pass, in f32: a change
    of 2^-6 in one entry, whose second-order term the central difference cancels and whose third
    is below 2^-18 times the third derivative (of order 1), over sums of 40 f32 values of
    magnitude 3 that are off by 2^-20 each: 2^-14 / 2^-6 at most together, 0.02 allowed."""
    rng = rng_of(15, kind)
    M, N, h = 2, 20, 2.0 ** -6
    k = Z.ZERO_NORM_LAYER if kind == "layer" else Z.ZERO_NORM_RMS
    x, dy = (torch.from_numpy(rand(rng, M, N)).to(dev()) for _ in range(2))
    w, b = vec(rng, N, 1.0), vec(rng, N)

    def loss(x, w, b):
        return float((dy.double() * Z.zero_norm_forward(x, w, b, kind=k, dtype=F32).double()).sum())

    st = Z.zero_norm_forward(x, w, b, kind=k, stats=True)[1]
    dw, db = torch.empty(N, device=dev()), torch.empty(N, device=dev())
    dx = Z.zero_norm_grad(dy, x, w, st, kind=k, dweight=dw, dbias=db)
    for i in range(M):
        for j in range(N):
            up, down = x.clone(), x.clone()
            up[i, j] += h
            down[i, j] -= h
            diff = (loss(up, w, b) - loss(down, w, b)) / float(up[i, j].double() - down[i, j].double())
            assert abs(diff - float(dx[i, j])) < 0.02
    for t, got in ((w, dw), (b, db)):
        for j in range(N):
            up, down = t.clone(), t.clone()
            up[j] += 0.25
            down[j] -= 0.25
            args = [(x, up, b), (x, down, b)] if t is w else [(x, w, up), (x, w, down)]
            diff = (loss(*args[0]) - loss(*args[1])) / float(up[j].double() - down[j].double())
            assert abs(diff - float(got[j])) < 0.02


def test_same_call_same_bits(Z):
    """The weight's gradient does not depend on timing."""
    rng = rng_of(16)
    for M, N in ((5000, 768), (3000, 2000), (40, 20000)):
        dy, x = (torch.from_numpy(rand(rng, M, N)).to(dev()).to(BF) for _ in range(2))
        st = Z.zero_norm_forward(x, stats=True)[1]
        got = []
        for _ in range(3):
            dw, db = torch.empty(N, device=dev()), torch.empty(N, device=dev())
            got.append((Z.zero_norm_grad(dy, x, None, st, dweight=dw, dbias=db), dw, db))
        assert all(torch.equal(p, q) for g in got[1:] for p, q in zip(g, got[0]))


def test_streams_and_graphs(Z):
    """Calls on a stream of their own, two at a time with workspaces of their own, and
    captured and replayed on new inputs between the program's own work."""
    rng = rng_of(17)
    M, N = 600, 1000
    xs, dys = ([torch.from_numpy(rand(rng, M, N)).to(dev()).to(BF) for _ in range(2)] for _ in range(2))
    w = vec(rng, N, 1.0)

    def run(x, dy, dw, db, stream=None):
        y, st = Z.zero_norm_forward(x, w, stats=True, stream=stream)
        return y, Z.zero_norm_grad(dy, x, w, st, dweight=dw, dbias=db, stream=stream), dw, db

    def new():
        return torch.empty(N, device=dev()), torch.empty(N, device=dev())

    want = [run(x, dy, *new()) for x, dy in zip(xs, dys)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs = [new() for _ in range(2)]
    got = [run(x, dy, *o, stream=s) for x, dy, o, s in zip(xs, dys, outs, streams)]
    torch.cuda.synchronize()
    for g, v in zip(got, want):
        assert all(torch.equal(p, q) for p, q in zip(g, v))
    x, dy, o = xs[0].clone(), dys[0].clone(), new()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = run(x, dy, *o)
    for k in (1, 0, 1):
        x.copy_(xs[k])
        dy.copy_(dys[k])
        o[0].zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(captured, want[k]))


def test_many_rows(Z):
    """More rows than one launch of a wave each would count bytes of in 32 bits."""
    M, N = 3_000_000, 400
    g = torch.Generator(device=dev()).manual_seed(3)
    x = torch.empty(M, N, dtype=BF, device=dev()).normal_(generator=g)
    y, st = Z.zero_norm_forward(x, stats=True)
    dw = torch.empty(N, device=dev())
    dx = Z.zero_norm_grad(x, x, None, st, dweight=dw)
    pick = torch.tensor([0, 1, M // 2, M - 2, M - 1], device=dev())
    s64 = x[pick].cpu().double().numpy()
    want, err, stats, es = R.forward(s64, np.ones(N), np.zeros(N), rms=False, eps=1e-5, out="bf16")
    close("y", y[pick], want, err)
    close("stats", st[pick], stats, es)
    close("dx", dx[pick], *R.grad(s64, s64, np.ones(N), st[pick].cpu().double().numpy(), rms=False)[0])
    # the mean over the columns of dw = sum of x (x - mean) rstd is the sum over the rows of var rstd,
    # var = 1 / rstd^2 - eps. A wave adds 3,000,000 / 4,096 rows in a chain, then at most 60 partial
    # sums: 800 * 2^-24 < 5e-5 of the sum of magnitudes, which is the sum itself but for a hundredth
    r = st[:, 1].double()
    want = float(((r ** -2 - 1e-5) * r).sum())
    assert abs(float(dw.double().mean()) / want - 1.0) < 1e-4


def test_refuses(Z):
    x = torch.zeros(4, 8, dtype=BF, device=dev())
    st = torch.zeros(4, 2, device=dev())
    f, g = Z.zero_norm_forward, Z.zero_norm_grad
    for call, word in ((lambda: f(x.half()), "neither"), (lambda: f(x[0]), "shape"), (lambda: f(x.t()), "stride"),
                       (lambda: f(x, torch.ones(7, dtype=BF, device=dev())), "weight"),
                       (lambda: f(x, torch.ones(8, device=dev())), "weight"),
                       (lambda: f(x, sum=x), "without a residual"),
                       (lambda: f(x, residual=x[:3]), "residual has shape"),
                       (lambda: f(x, stats=torch.zeros(4, 3, device=dev())), "stats"),
                       (lambda: f(x, stats=torch.zeros(4, 4, device=dev())[:, :2]), "stats has row stride"),
                       (lambda: f(x, y=x.float(), dtype=BF), "y is"),
                       (lambda: f(x, eps=-1.0), "eps"), (lambda: f(x, kind=4), "kind"),
                       (lambda: f(x, y=x.view(-1)[1:25].view(3, 8)), "y has shape"),
                       (lambda: g(x, x), "stats"), (lambda: g(x, x[:, :4], None, st), "x has shape"),
                       (lambda: g(x, x, None, st, residual_grad=x.float(), dtype=BF), "residual_grad"),
                       (lambda: g(x, x, None, st, dweight=torch.zeros(8, dtype=BF, device=dev()),
                                  dbias=torch.zeros(8, device=dev())), "dbias"),
                       (lambda: g(x, x, None, st, dweight=torch.zeros(8, device=dev()),
                                  workspace=torch.zeros(4, device=dev())), "ws_bytes"),
                       (lambda: f(x, residual=x, y=x, sum=x), "overlap")):
        say("refused for", word)
        with pytest.raises(Z.ZeroError, match=word):
            call()


@pytest.mark.parametrize("N", [12, 100, 1000])
def test_grad_of_a_row_far_from_zero(Z, N):
    """Equal elements so large that mean times 1/sigma passes fp32: h is 0 in every column, and
    the columns behind the last add nothing (not 0 times an infinity). The norm of a row of
    2^118 is exact, and so 1/sigma is eps^-1/2; dx is rstd (dy - mean(dy)) in fp32 with at
    most 2 N + 8 roundings of 2^-24 of at most max |dy| each, before bf16's."""
    M = 5
    dy = torch.randn(M, N, generator=torch.Generator().manual_seed(N)).to(dev()).bfloat16()
    x = torch.full((M, N), 2.0 ** 118, device=dev())
    say("far from zero", N)
    y, stats = Z.zero_norm_forward(x, kind=Z.ZERO_NORM_LAYER, eps=1e-12, stats=True)
    assert bool((y == 0).all()) and bool((stats[:, 0] == 2.0 ** 118).all())
    for xt in (x, x.bfloat16()):
        dw, db = (torch.zeros(N, device=dev()) for _ in range(2))
        dx = Z.zero_norm_grad(dy, xt, None, stats, kind=Z.ZERO_NORM_LAYER, dtype=torch.float32, dweight=dw, dbias=db)
        want = 1e6 * (dy.double() - dy.double().mean(1, keepdim=True))
        assert float((dx.double() - want).abs().max()) <= 1e6 * (2 * N + 8) * 2.0 ** -24 * float(dy.double().abs().max())
        assert bool((dw == 0).all())
        assert float((db.double() - dy.double().sum(0)).abs().max()) <= 8 * M * 2.0 ** -24 * float(dy.double().abs().max())
