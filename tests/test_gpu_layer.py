"""GPU tests of the layer operators against tests/layer_ref.py in 64 bits.

Every matrix of a case lies in a larger buffer: rows longer than their columns,
a base at any element, NaN in what inputs leave unused and a sentinel in what
outputs must not touch. The bounds are worst-case ones of fp32 sums and a single
rounding, derived in layer_ref.py.
"""
import zlib

import numpy as np
import pytest
import torch

import layer_ref as R
from gpu_util import dev, say

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32
TY = {"bf16": BF, "f32": F32}
SENT = -12345.0                     # exact in both types


class Mat:
    """A matrix inside a larger buffer."""

    def __init__(self, rows, cols, dtype, *, ld=None, shift=0, fill=None, pad=SENT):
        self.rows, self.cols = rows, cols
        self.ld = ld = cols if ld is None else ld
        n = rows * ld + shift + 64
        self.raw = torch.full((n + 64,), pad, dtype=dtype, device=dev())
        self.t = self.raw[64 + shift:64 + shift + rows * ld].view(rows, ld)[:, :cols] if rows and ld else \
            torch.empty((rows, cols), dtype=dtype, device=dev())
        if fill is not None and self.t.numel():
            self.t.copy_(torch.from_numpy(fill))
        self.before = self.raw.clone()

    def f64(self):
        return self.t.cpu().double().numpy()

    def intact_outside(self):
        """Nothing outside the matrix has changed."""
        m = torch.zeros_like(self.raw, dtype=torch.bool)
        if self.t.numel():
            off = self.t.storage_offset()
            m[off:off + self.rows * self.ld].view(self.rows, self.ld)[:, :self.cols] = True
        a, b = self.raw, self.before
        same = (a == b) | (a.isnan() & b.isnan())
        return bool((same | m).all())


def rand(rng, *shape, scale=1.0):
    return (rng.standard_normal(shape) * scale).astype(np.float32)


def rng_of(case):
    """A generator of its own for each case, the same in every run."""
    return np.random.default_rng(zlib.crc32(repr(case).encode()))


def inp(rng, rows, cols, *, dtype=BF, scale=1.0, pad_ld=0, shift=0):
    return Mat(rows, cols, dtype, ld=cols + pad_ld, shift=shift, fill=rand(rng, rows, cols, scale=scale),
               pad=float("nan"))


def close(name, got, want, err):
    got = got.cpu().double().numpy()
    assert got.shape == want.shape
    d = np.abs(got - want)
    bad = ~(d <= err)
    if bad.any():
        i = tuple(int(x) for x in np.argwhere(bad)[0])
        raise AssertionError(f"{name}: {int(bad.sum())} of {bad.size} off; at {i} got {got[i]!r}, want {want[i]!r}, "
                             f"allowed {err[i]!r}")


# (M, K, N): single rows, lengths of zero and one, edges of the 16, 64, 128 and 256 tiles,
# odd sizes, long reductions that are split, wide outputs
SIZES = [(1, 1, 1), (1, 768, 2304), (2, 7, 9), (3, 0, 5), (5, 8, 1), (1, 64, 8), (16, 32, 16), (17, 33, 31),
         (63, 64, 65), (64, 128, 64), (127, 129, 128), (128, 64, 256), (130, 200, 257), (255, 511, 129),
         (257, 96, 384), (300, 1000, 72), (33, 4096, 40), (4, 2500, 700), (512, 320, 512), (1000, 72, 130),
         (1, 5000, 3), (40, 1, 520)]
LAYOUTS = [0, 1]
# (rows' extra length, base shift in elements): aligned rows, padded aligned rows, odd rows, odd base
PLACES = [(0, 0), (8, 0), (1, 0), (0, 1), (5, 3)]


def weight(rng, K, N, layout, place, scale=0.1):
    r, c = (N, K) if layout == 0 else (K, N)
    return inp(rng, r, c, scale=scale, pad_ld=place[0], shift=place[1])


def w64(w, layout):
    return w.f64() if layout == 0 else w.f64().T


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_forward_sizes(Z, size, layout):
    M, K, N = size
    rng = rng_of((1,) + size + (layout,))
    place = PLACES[(M + K + N) % len(PLACES)]
    x, w = inp(rng, M, K, pad_ld=place[0], shift=place[1]), weight(rng, K, N, layout, place)
    b = torch.from_numpy(rand(rng, N)).to(dev()).to(BF)
    y, z = (Mat(M, N, BF, ld=N + place[0], shift=place[1]) for _ in range(2))
    say("forward", size, layout, place)
    Z.zero_linear_forward(x.t, w.t, b, w_layout=layout, y=y.t, preact=z.t)
    want, err, wz, ez = R.linear_forward(x.f64(), w64(w, layout), b.cpu().double().numpy())
    close("y", y.t, want, err)
    close("z", z.t, wz, ez)
    assert y.intact_outside() and z.intact_outside()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("size", SIZES, ids=str)
def test_grad_input_sizes(Z, size, layout):
    M, K, N = size
    rng = rng_of((2,) + size + (layout,))
    place = PLACES[(M + K + 2 * N) % len(PLACES)]
    dz, w = inp(rng, M, N, pad_ld=place[0], shift=place[1]), weight(rng, K, N, layout, place)
    dx = Mat(M, K, F32, ld=K + place[0], shift=place[1])
    say("grad input", size, layout, place)
    Z.zero_linear_grad_input(dz.t, w.t, w_layout=layout, dx=dx.t)
    want, err = R.linear_grad_input(dz.f64(), w64(w, layout), out="f32")
    close("dx", dx.t, want, err)
    assert dx.intact_outside()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("size", SIZES + [(0, 5, 7), (4000, 128, 96), (8200, 24, 136), (2049, 130, 1)], ids=str)
def test_grad_weight_sizes(Z, size, layout):
    M, K, N = size
    rng = rng_of((3,) + size + (layout,))
    place = PLACES[(2 * M + K + N) % len(PLACES)]
    out = ("bf16", "f32")[(M + N) % 2]
    accumulate = bool((M + K) % 2)
    dz, x = inp(rng, M, N, pad_ld=place[0], shift=place[1]), inp(rng, M, K, pad_ld=place[0], shift=place[1])
    r, c = (N, K) if layout == 0 else (K, N)
    dw = Mat(r, c, TY[out], ld=c + place[0], shift=place[1], fill=rand(rng, r, c))
    db = Mat(1, N, TY[out], shift=place[1], fill=rand(rng, 1, N))
    old_w, old_b = w64(dw, layout), db.f64()[0]
    say("grad weight", size, layout, place, out, accumulate)
    Z.zero_linear_grad_weight(dz.t, x.t, dw.t, db.t.reshape(-1), w_layout=layout, accumulate=accumulate)
    want, err = R.linear_grad_weight(dz.f64(), x.f64(), old=old_w if accumulate else None, out=out)
    close("dw", dw.t if layout == 0 else dw.t.t(), want, err)
    want, err = R.column_sums(dz.f64(), old=old_b if accumulate else None, out=out)
    close("db", db.t[0], want, err)
    assert dw.intact_outside() and db.intact_outside()


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("act", range(4))
@pytest.mark.parametrize("size", [(1, 64, 72), (37, 40, 203), (256, 128, 512), (5, 3000, 260)], ids=str)
def test_forward_epilogue(Z, size, act, out):
    M, K, N = size
    rng = rng_of((4,) + size + (act,))
    layout, place = act % 2, PLACES[(act + M) % len(PLACES)]
    p, seed, offset = (0.0, 0.1, 0.5, 1 - 2.0 ** -16)[(act + N) % 4], 0xFEDCBA9876543210 + act, (1 << 63) + 5
    x, w = inp(rng, M, K, pad_ld=place[0], shift=place[1]), weight(rng, K, N, layout, place, 0.3)
    b = torch.from_numpy(rand(rng, N)).to(dev()).to(BF)
    res = inp(rng, M, N, dtype=TY[out], pad_ld=place[0], shift=place[1])
    y, z = Mat(M, N, TY[out], ld=N + place[0]), Mat(M, N, BF, ld=N + place[0])
    say("forward epilogue", size, act, out, p)
    Z.zero_linear_forward(x.t, w.t, b, w_layout=layout, act=act, dropout=Z.zero_dropout(p, seed, offset),
                          residual=res.t, y=y.t, preact=z.t)
    want, err, wz, ez = R.linear_forward(x.f64(), w64(w, layout), b.cpu().double().numpy(), act_name=R.ACTS[act],
                                         p=p, seed=seed, offset=offset, residual=res.f64(), out=out)
    close("y", y.t, want, err)
    close("z", z.t, wz, ez)
    assert y.intact_outside() and z.intact_outside()
    # in place over the residual, and without the rest of the epilogue's outputs
    Z.zero_linear_forward(x.t, w.t, b, w_layout=layout, act=act, dropout=Z.zero_dropout(p, seed, offset),
                          residual=res.t, y=res.t)
    assert torch.equal(res.t, y.t)


@pytest.mark.parametrize("out", ["bf16", "f32"])
@pytest.mark.parametrize("act", range(4))
@pytest.mark.parametrize("size", [(1, 72, 64), (37, 203, 40), (256, 512, 128), (5, 260, 3000)], ids=str)
def test_grad_input_epilogue(Z, size, act, out):
    M, K, N = size
    rng = rng_of((5,) + size + (act,))
    layout, place = act % 2, PLACES[(act + M + 1) % len(PLACES)]
    p, seed, offset = (0.3, 0.0, 0.7, 0.1)[(act + N) % 4], 77 + act, 1 << 40
    dz, w = inp(rng, M, N, pad_ld=place[0], shift=place[1]), weight(rng, K, N, layout, place)
    z = inp(rng, M, K, scale=3.0, pad_ld=place[0], shift=place[1])
    dx = Mat(M, K, TY[out], ld=K + place[0])
    say("grad input epilogue", size, act, out, p)
    Z.zero_linear_grad_input(dz.t, w.t, w_layout=layout, act=act, preact=z.t,
                             dropout=Z.zero_dropout(p, seed, offset), dx=dx.t)
    want, err = R.linear_grad_input(dz.f64(), w64(w, layout), act_name=R.ACTS[act], z=z.f64(), p=p, seed=seed,
                                    offset=offset, out=out)
    close("dx", dx.t, want, err)
    assert dx.intact_outside()
    if out == "bf16":
        Z.zero_linear_grad_input(dz.t, w.t, w_layout=layout, act=act, preact=z.t,
                                 dropout=Z.zero_dropout(p, seed, offset), dx=z.t)
        assert torch.equal(z.t, dx.t)


DROP_SIZES = [(1, 1), (1, 7), (3, 8), (5, 9), (64, 768), (17, 1003), (300, 64), (2, 40000), (70000, 3)]


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")], ids=str)
@pytest.mark.parametrize("size", DROP_SIZES, ids=str)
def test_dropout_add(Z, size, types):
    M, N = size
    rng = rng_of((6,) + size)
    place = PLACES[(M + N) % len(PLACES)]
    p, seed, offset = (0.1, 0.5, 0.9, 0.0)[(M + len(types[0])) % 4], 1 << 33 | M, N
    x = inp(rng, M, N, dtype=TY[types[0]], pad_ld=place[0], shift=place[1])
    res = inp(rng, M, N, dtype=TY[types[1]], pad_ld=place[0], shift=place[1])
    y = Mat(M, N, TY[types[1]], ld=N + place[0], shift=place[1])
    drop = Z.zero_dropout(p, seed, offset)
    say("dropout add", size, types, p)
    for r in (None, res):
        Z.zero_dropout_add(x.t, drop, residual=None if r is None else r.t, y=y.t)
        want, err = R.dropout_add(x.f64(), p=p, seed=seed, offset=offset, residual=None if r is None else r.f64(),
                                  out=types[1])
        close("y", y.t, want, err)
        assert y.intact_outside()
    Z.zero_dropout_add(x.t, drop, residual=res.t, y=res.t)
    assert torch.equal(res.t, y.t)
    if types[0] == types[1]:
        want = Z.zero_dropout_add(x.t, drop)
        Z.zero_dropout_add(x.t, drop, y=x.t)
        assert torch.equal(x.t, want)


@pytest.mark.parametrize("types", [("bf16", "bf16"), ("f32", "f32"), ("bf16", "f32"), ("f32", "bf16")], ids=str)
@pytest.mark.parametrize("act", range(4))
@pytest.mark.parametrize("size", DROP_SIZES[:7], ids=str)
def test_dropout_grad(Z, size, act, types):
    M, N = size
    rng = rng_of((7,) + size + (act,))
    place = PLACES[(M + N + act) % len(PLACES)]
    p, seed, offset = (0.25, 0.0, 0.5)[(M + act) % 3], 3, 1 << 62
    dy = inp(rng, M, N, dtype=TY[types[0]], pad_ld=place[0], shift=place[1])
    z = inp(rng, M, N, scale=4.0, pad_ld=place[0], shift=place[1])
    dz = Mat(M, N, TY[types[1]], ld=N + place[0], shift=place[1])
    say("dropout grad", size, act, types, p)
    Z.zero_dropout_grad(dy.t, Z.zero_dropout(p, seed, offset), act=act, preact=z.t, dz=dz.t)
    want, err = R.dropout_grad(dy.f64(), p=p, seed=seed, offset=offset, act_name=R.ACTS[act], z=z.f64(), out=types[1])
    close("dz", dz.t, want, err)
    assert dz.intact_outside()


def test_masks_agree_everywhere(Z):
    """The product's epilogue, its gradient's and the two elementwise calls drop the
    same elements of a matrix, whatever its place."""
    M, K, N = 150, 96, 333
    rng = np.random.default_rng(8)
    drop = Z.zero_dropout(0.4, 1234567890123, 42)
    want = R.drop_factor(M, N, 0.4, 1234567890123, 42) != 0
    x = inp(rng, M, K)
    w = torch.zeros((N, K), dtype=BF, device=dev())
    one = torch.ones(N, dtype=BF, device=dev())
    got = [Z.zero_linear_forward(x.t, w, one, dropout=drop),
           Z.zero_dropout_add(torch.ones((M, N), dtype=F32, device=dev()), drop),
           Z.zero_dropout_grad(torch.ones((M, N), dtype=BF, device=dev()), drop)]
    eye = torch.eye(N, dtype=BF, device=dev())
    got.append(Z.zero_linear_grad_input(torch.ones((M, N), dtype=BF, device=dev()), eye, dropout=drop))
    for g in got:
        assert np.array_equal((g != 0).cpu().numpy(), want)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_nonfinite_values(Z, bad):
    """A NaN or infinity reaches exactly the outputs that its row or column feeds, none
    behind a dropped element, and large finite pre-activations have finite slopes."""
    M, K, N = 70, 72, 130
    rng = np.random.default_rng(9)
    x, w = inp(rng, M, K), inp(rng, N, K)
    x.t[3, 5] = bad
    w.t[7, 71] = bad
    y = Z.zero_linear_forward(x.t, w.t, dtype=F32)
    want = torch.zeros((M, N), dtype=torch.bool)
    want[3, :] = True
    want[:, 7] = True
    assert torch.equal(~torch.isfinite(y).cpu(), want)
    drop = Z.zero_dropout(0.5, 3, 4)
    keep = torch.from_numpy(R.drop_factor(M, N, 0.5, 3, 4) != 0)
    y = Z.zero_linear_forward(x.t, w.t, dropout=drop)
    assert torch.equal(~torch.isfinite(y).cpu(), want & keep)
    full = torch.full((M, N), bad, dtype=BF, device=dev())
    y = Z.zero_dropout_add(full, drop)
    assert torch.equal(~torch.isfinite(y).cpu(), keep)
    assert bool((y[~keep.to(dev())] == 0).all())
    dz = Z.zero_dropout_grad(full, drop, act=2, preact=torch.ones((M, N), dtype=BF, device=dev()))
    assert torch.equal(~torch.isfinite(dz).cpu(), keep)
    dw = torch.zeros((N, K), dtype=F32, device=dev())
    d2 = inp(rng, M, N)
    Z.zero_linear_grad_weight(d2.t, x.t, dw)
    want = torch.zeros((N, K), dtype=torch.bool)
    want[:, 5] = True
    assert torch.equal(~torch.isfinite(dw).cpu(), want)
    big = torch.tensor([[3e38, -3e38, 1e20, -1e20, 40.0, -40.0, 0.0, float("inf")]], dtype=BF, device=dev())
    one = torch.ones((1, 8), dtype=F32, device=dev())
    for act in (1, 2, 3):
        s = Z.zero_dropout_grad(one, None, act=act, preact=big, dtype=F32).cpu()[0]
        half = 0.0 if act == 1 else 0.5
        assert torch.equal(s, torch.tensor([1.0, 0, 1, 0, 1, 0, half, 1.0]) if act == 1 else s)
        assert torch.allclose(s, torch.tensor([1.0, 0, 1, 0, 1, 0, half, 1.0]), atol=1e-12)


def test_past_32_bits(Z):
    """Rows so far apart that element offsets pass 2^31 and byte offsets 2^32."""
    M, K, N, ld = 2100, 40, 64, 1 << 20
    rng = np.random.default_rng(10)
    raw = torch.zeros(M * ld, dtype=BF, device=dev())
    x = raw.view(M, ld)[:, 16:16 + K]
    x.copy_(torch.from_numpy(rand(rng, M, K)))
    w = inp(rng, N, K)
    y = raw.view(M, ld)[:, 128:128 + N]
    Z.zero_linear_forward(x, w.t, y=y)
    want, err, _, _ = R.linear_forward(x.cpu().double().numpy(), w.f64())
    close("y", y, want, err)
    dw = torch.zeros((N, K), dtype=F32, device=dev())
    db = torch.zeros(N, dtype=F32, device=dev())
    Z.zero_linear_grad_weight(y, x, dw, db)
    want, err = R.linear_grad_weight(y.cpu().double().numpy(), x.cpu().double().numpy(), out="f32")
    close("dw", dw, want, err)
    want, err = R.column_sums(y.cpu().double().numpy(), out="f32")
    close("db", db, want, err)
    dx = raw.view(M, ld)[:, 512:512 + K]
    Z.zero_linear_grad_input(y, w.t, dx=dx)
    want, err = R.linear_grad_input(y.cpu().double().numpy(), w.f64())
    close("dx", dx, want, err)
    d = raw.view(M, ld)[:, 1024:1024 + N]
    Z.zero_dropout_add(y, Z.zero_dropout(0.5, 1, 2), y=d)
    want, err = R.dropout_add(y.cpu().double().numpy(), p=0.5, seed=1, offset=2)
    close("d", d, want, err)


def test_repeated_calls_are_bitwise_equal(Z):
    """The splits of a long sum are joined in a fixed order."""
    rng = np.random.default_rng(11)
    M, K, N = 5000, 136, 264
    dz, x = inp(rng, M, N), inp(rng, M, K)
    outs = []
    for _ in range(3):
        dw = torch.zeros((N, K), dtype=F32, device=dev())
        db = torch.zeros(N, dtype=F32, device=dev())
        Z.zero_linear_grad_weight(dz.t, x.t, dw, db)
        y = Z.zero_linear_forward(dz.t[:9], dw.to(BF), w_layout=1)
        outs.append((dw, db, y))
    for o in outs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(o, outs[0]))


def test_streams_and_workspaces(Z):
    """Calls on two streams, with workspaces of their own, given or allocated."""
    rng = np.random.default_rng(12)
    M, K, N = 4096, 128, 192
    need = Z.zero_linear_workspace_bytes(Z.ZERO_LINEAR_GRAD_WEIGHT, 0, M, K, N)
    assert need > 0
    data = [(inp(rng, M, N), inp(rng, M, K)) for _ in range(2)]
    want = []
    for dz, x in data:
        dw = torch.zeros((N, K), dtype=F32, device=dev())
        Z.zero_linear_grad_weight(dz.t, x.t, dw)
        want.append(dw)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    ws = [torch.empty(need, dtype=torch.uint8, device=dev()) for _ in range(2)]
    got = [torch.zeros((N, K), dtype=F32, device=dev()) for _ in range(2)]
    torch.cuda.synchronize()
    for _ in range(5):
        for k in range(2):
            Z.zero_linear_grad_weight(data[k][0].t, data[k][1].t, got[k], workspace=ws[k], stream=streams[k])
        for k in range(2):
            Z.zero_linear_grad_weight(data[k][0].t, data[k][1].t, got[k], stream=streams[k])
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    with pytest.raises(Z.ZeroError) as e:
        Z.zero_linear_grad_weight(data[0][0].t, data[0][1].t, got[0], workspace=ws[0][:16])
    assert e.value.status == -3


def test_refusals_of_tensors(Z):
    a = torch.zeros((4, 8), dtype=BF, device=dev())
    for bad in (lambda: Z.zero_linear_forward(a.t(), a), lambda: Z.zero_linear_forward(a, a[:, :7]),
                lambda: Z.zero_linear_forward(a, a.cpu()), lambda: Z.zero_linear_forward(a.float(), a),
                lambda: Z.zero_linear_forward(a, a, torch.zeros(5, dtype=BF, device=dev())),
                lambda: Z.zero_linear_forward(a, a, dtype=torch.float16),
                lambda: Z.zero_linear_forward(a, a, w_layout=3),
                lambda: Z.zero_linear_forward(a[0].expand(4, 8), a),
                lambda: Z.zero_linear_grad_input(a, a.t().contiguous(), act=1),
                lambda: Z.zero_linear_grad_weight(a, a[:3], a),
                lambda: Z.zero_dropout_add(a.half(), None),
                lambda: Z.zero_dropout_grad(a, Z.zero_dropout(1.5)),
                lambda: Z.zero_dropout(0.5, counter=torch.zeros(1, dtype=torch.int32, device=dev())),
                lambda: Z.zero_linear_forward(a, a, y=a[:, :4])):
        with pytest.raises(Z.ZeroError):
            bad()


def test_captured_calls_draw_anew(Z):
    """A captured forward and backward with the device counter: every replay equals the
    eager calls at the same counter, with eager work between replays."""
    rng = np.random.default_rng(13)
    M, K, N = 192, 256, 136
    x, w = inp(rng, M, K), inp(rng, N, K, scale=0.1)
    dy = inp(rng, M, N)
    counter = torch.zeros(1, dtype=torch.int64, device=dev())
    drop = Z.zero_dropout(0.3, 5, 100, counter=counter)
    y = torch.empty((M, N), dtype=BF, device=dev())
    z, dz, dx = torch.empty_like(y), torch.empty_like(y), torch.empty((M, K), dtype=BF, device=dev())
    dw = torch.zeros((N, K), dtype=F32, device=dev())
    db = torch.zeros(N, dtype=F32, device=dev())
    ws = torch.empty(max(Z.zero_linear_workspace_bytes(k, 0, M, K, N) for k in range(3)), dtype=torch.uint8,
                     device=dev())

    def calls(drop, y, z, dz, dx, dw, db, ws):
        Z.zero_linear_forward(x.t, w.t, act=2, dropout=drop, y=y, preact=z, workspace=ws)
        Z.zero_dropout_grad(dy.t, drop, act=2, preact=z, dz=dz)
        Z.zero_linear_grad_weight(dz, x.t, dw, db, accumulate=True, workspace=ws)
        Z.zero_linear_grad_input(dz, w.t, dx=dx, workspace=ws)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        calls(drop, y, z, dz, dx, dw, db, ws)
        torch.cuda.synchronize()
        dw.zero_(), db.zero_()
        with torch.cuda.graph(graph, stream=s):
            calls(drop, y, z, dz, dx, dw, db, ws)
    torch.cuda.synchronize()
    e = [torch.zeros_like(t) for t in (y, z, dz, dx, dw, db)]
    masks = []
    for k in range(4):
        counter.fill_(7 * k)
        graph.replay()
        torch.cuda.synchronize()
        calls(Z.zero_dropout(0.3, 5, 100 + 7 * k), *e, torch.empty_like(ws))
        torch.cuda.synchronize()
        for name, a, b in zip("y z dz dx dw db".split(), (y, z, dz, dx, dw, db), e):
            assert torch.equal(a, b), (k, name)
        masks.append(y == 0)
    assert not torch.equal(masks[0], masks[1])


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("rows,inner", [(4100, 136), (4096, 64), (4345, 191), (4097, 320)])
def test_wide_outputs(Z, rows, inner, layout):
    """Outputs of enough tiles to fill the chip (the largest tiles), with ragged edges
    and reductions that are and are not whole tiles, in each direction."""
    rng = rng_of((14, rows, inner, layout))
    cols = 4104
    say("wide", rows, inner, layout)
    x, w = inp(rng, rows, inner, pad_ld=-inner % 8), weight(rng, inner, cols, layout, (8, 0))
    res = inp(rng, rows, cols)
    y, z = Mat(rows, cols, BF, ld=cols + 8), Mat(rows, cols, BF, ld=cols + 16)
    Z.zero_linear_forward(x.t, w.t, w_layout=layout, act=2, dropout=Z.zero_dropout(0.2, 1, 2), residual=res.t, y=y.t,
                          preact=z.t)
    want, err, wz, ez = R.linear_forward(x.f64(), w64(w, layout), act_name="gelu", p=0.2, seed=1, offset=2,
                                         residual=res.f64())
    close("y", y.t, want, err)
    close("z", z.t, wz, ez)
    assert y.intact_outside() and z.intact_outside()
    dz, w = inp(rng, rows, inner, pad_ld=-inner % 8), weight(rng, cols, inner, layout, (-inner % 8, 0))
    dx = Mat(rows, cols, F32, ld=cols + 8)
    Z.zero_linear_grad_input(dz.t, w.t, w_layout=layout, act=3, preact=res.t, dx=dx.t)
    want, err = R.linear_grad_input(dz.f64(), w64(w, layout), act_name="silu", z=res.f64(), out="f32")
    close("dx", dx.t, want, err)
    assert dx.intact_outside()
    dz, x = inp(rng, inner, rows, pad_ld=-rows % 8), inp(rng, inner, cols)
    r, c = (rows, cols) if layout == 0 else (cols, rows)
    dw = Mat(r, c, F32, ld=c + 8, fill=rand(rng, r, c))
    old = w64(dw, layout)
    Z.zero_linear_grad_weight(dz.t, x.t, dw.t, w_layout=layout, accumulate=True)
    want, err = R.linear_grad_weight(dz.f64(), x.f64(), old=old, out="f32")
    close("dw", dw.t if layout == 0 else dw.t.t(), want, err)
    assert dw.intact_outside()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("M,K,N", [(70, 4104, 4100), (512, 16, 4200), (333, 4200, 8), (9000, 264, 260), (64, 2048, 2304),
                                   (100, 0, 300)])
def test_bias_gradient_of_wide_weights(Z, M, K, N, layout):
    """The bias gradient beside weight gradients of many tiles, of one row or column of
    tiles, of split sums, and of a weight with no elements."""
    rng = rng_of((15, M, K, N, layout))
    say("bias", M, K, N, layout)
    dz, x = inp(rng, M, N, pad_ld=-N % 8), inp(rng, M, K, pad_ld=-K % 8)
    r, c = (N, K) if layout == 0 else (K, N)
    dw = torch.zeros((r, c), dtype=F32, device=dev())
    db = Mat(1, N, F32, fill=rand(rng, 1, N))
    old = db.f64()[0]
    Z.zero_linear_grad_weight(dz.t, x.t, dw, db.t[0], w_layout=layout, accumulate=True)
    want, err = R.column_sums(dz.f64(), old=old, out="f32")
    close("db", db.t[0], want, err)
    assert db.intact_outside()
    want, err = R.linear_grad_weight(dz.f64(), x.f64(), out="f32")
    close("dw", dw if layout == 0 else dw.t(), want, err)


@pytest.mark.parametrize("M,K,N", [(4352, 72, 4096), (4096, 192, 4608), (2048, 64, 16640), (8192, 128, 2304)])
def test_rounds_and_quarters(Z, M, K, N):
    """Tile counts a little over whole rounds of the chip, whose rest goes to smaller
    tiles, in a second launch."""
    rng = np.random.default_rng(16 + M)
    x, w = inp(rng, M, K), inp(rng, N, K, scale=0.1)
    y = Mat(M, N, BF, ld=N + 8)
    Z.zero_linear_forward(x.t, w.t, y=y.t)
    want, err, _, _ = R.linear_forward(x.f64(), w.f64())
    close("y", y.t, want, err)
    assert y.intact_outside()
    dz = inp(rng, K, M)
    dw = torch.empty((M, N), dtype=BF, device=dev())
    db = torch.empty(M, dtype=BF, device=dev())
    x = inp(rng, K, N)
    Z.zero_linear_grad_weight(dz.t, x.t, dw, db)
    want, err = R.linear_grad_weight(dz.f64(), x.f64())
    close("dw", dw, want, err)
    want, err = R.column_sums(dz.f64())
    close("db", db, want, err)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("M,K,N", [(1, 768, 2304), (2, 2304, 768), (4, 4100, 515), (7, 71, 4096), (15, 640, 200),
                                   (16, 4096, 1100), (16, 63, 17), (17, 768, 768), (1, 2, 3000), (3, 11008, 64)])
def test_few_rows(Z, M, K, N, layout):
    """One to seventeen rows: the products that are bound by the weights' bytes, with
    the whole epilogue, whole and odd reductions, padded and odd rows."""
    rng = rng_of((17, M, K, N, layout))
    for place in ((0, 0), (8, 0), (3, 1)):
        x, w = inp(rng, M, K, pad_ld=place[0], shift=place[1]), weight(rng, K, N, layout, place)
        b = torch.from_numpy(rand(rng, N)).to(dev()).to(BF)
        res = inp(rng, M, N)
        y, z = Mat(M, N, BF, ld=N + 5), Mat(M, N, BF, ld=N + 8)
        say("few rows", M, K, N, layout, place)
        Z.zero_linear_forward(x.t, w.t, b, w_layout=layout, act=3, dropout=Z.zero_dropout(0.25, 9, 8), residual=res.t,
                              y=y.t, preact=z.t)
        want, err, wz, ez = R.linear_forward(x.f64(), w64(w, layout), b.cpu().double().numpy(), act_name="silu", p=0.25,
                                             seed=9, offset=8, residual=res.f64())
        close("y", y.t, want, err)
        close("z", z.t, wz, ez)
        assert y.intact_outside() and z.intact_outside()
        dz = inp(rng, M, N, pad_ld=place[0], shift=place[1])
        zz = inp(rng, M, K)
        dx = Mat(M, K, F32, ld=K + 3)
        Z.zero_linear_grad_input(dz.t, w.t, w_layout=layout, act=2, preact=zz.t, dx=dx.t)
        want, err = R.linear_grad_input(dz.f64(), w64(w, layout), act_name="gelu", z=zz.f64(), out="f32")
        close("dx", dx.t, want, err)
        assert dx.intact_outside()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("rows,cols", [(8190, 765), (2900, 1530), (4097, 1152)])
@pytest.mark.parametrize("inner", [40, 200, 768])
def test_tiles_of_192_columns(Z, rows, cols, inner, layout):
    """Outputs of one round of the chip in tiles of 192 columns, of more in tiles of 128,
    with ragged edges, in each direction and type."""
    rng = rng_of((18, rows, cols, inner, layout))
    say("192", rows, cols, inner, layout)
    pad = -cols % 8
    x, w = inp(rng, rows, inner), weight(rng, inner, cols, layout, (pad if layout else 0, 0))
    res = inp(rng, rows, cols, pad_ld=3)
    y, z = Mat(rows, cols, BF, ld=cols + 5), Mat(rows, cols, BF, ld=cols + pad)
    b = inp(rng, 1, cols)
    Z.zero_linear_forward(x.t, w.t, b.t[0], w_layout=layout, act=3, dropout=Z.zero_dropout(0.3, 9, 8), residual=res.t,
                          y=y.t, preact=z.t)
    want, err, wz, ez = R.linear_forward(x.f64(), w64(w, layout), b.f64()[0], act_name="silu", p=0.3, seed=9, offset=8,
                                         residual=res.f64())
    close("y", y.t, want, err)
    close("z", z.t, wz, ez)
    assert y.intact_outside() and z.intact_outside()
    dz, w = inp(rng, rows, inner), weight(rng, cols, inner, layout, (0 if layout else pad, 0))
    dx = Mat(rows, cols, F32, ld=cols + 7)
    Z.zero_linear_grad_input(dz.t, w.t, w_layout=layout, act=2, preact=res.t, dropout=Z.zero_dropout(0.1, 2, 3), dx=dx.t)
    want, err = R.linear_grad_input(dz.f64(), w64(w, layout), act_name="gelu", z=res.f64(), p=0.1, seed=2, offset=3,
                                    out="f32")
    close("dx", dx.t, want, err)
    assert dx.intact_outside()
    r, c = (rows, cols) if layout == 0 else (cols, rows)
    dz, x = inp(rng, inner, rows, pad_ld=-rows % 8), inp(rng, inner, cols, pad_ld=pad)
    dw = Mat(r, c, BF, ld=c + 1, fill=rand(rng, r, c))
    old = w64(dw, layout)
    Z.zero_linear_grad_weight(dz.t, x.t, dw.t, w_layout=layout, accumulate=True)
    want, err = R.linear_grad_weight(dz.f64(), x.f64(), old=old)
    close("dw", dw.t if layout == 0 else dw.t.t(), want, err)
    assert dw.intact_outside()


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("rows,cols", [(8190, 2810), (2810, 8060)])
def test_rectangles(Z, rows, cols, layout):
    """Outputs whose last columns, or last rows, go to tiles of 192 columns in a launch
    behind the largest tiles', in each direction and with all that the epilogue takes."""
    rng = rng_of((20, rows, cols, layout))
    say("rectangles", rows, cols, layout)
    inner, pad = 968, -cols % 8
    x, w = inp(rng, rows, inner), weight(rng, inner, cols, layout, (pad if layout else 0, 0), 0.03)
    res, b, y = inp(rng, rows, cols, pad_ld=1), inp(rng, 1, cols), Mat(rows, cols, BF, ld=cols + 5)
    z = Mat(rows, cols, BF, ld=cols + 2)
    Z.zero_linear_forward(x.t, w.t, b.t[0], w_layout=layout, act=2, dropout=Z.zero_dropout(0.5, 4, 4), residual=res.t,
                          y=y.t, preact=z.t)
    want, err, wz, ez = R.linear_forward(x.f64(), w64(w, layout), b.f64()[0], act_name="gelu", p=0.5, seed=4, offset=4,
                                         residual=res.f64())
    close("y", y.t, want, err)
    close("z", z.t, wz, ez)
    assert y.intact_outside() and z.intact_outside()
    dz, w = inp(rng, rows, inner), weight(rng, cols, inner, layout, (0 if layout else pad, 0), 0.03)
    dx = Mat(rows, cols, BF, ld=cols + 7)
    Z.zero_linear_grad_input(dz.t, w.t, w_layout=layout, act=3, preact=res.t, dropout=Z.zero_dropout(0.2, 5, 5), dx=dx.t)
    want, err = R.linear_grad_input(dz.f64(), w64(w, layout), act_name="silu", z=res.f64(), p=0.2, seed=5, offset=5)
    close("dx", dx.t, want, err)
    assert dx.intact_outside()
    r, c = (rows, cols) if layout == 0 else (cols, rows)
    dz, x = inp(rng, inner, rows, pad_ld=-rows % 8), inp(rng, inner, cols, pad_ld=pad)
    for bias in (False, True):
        dw = Mat(r, c, F32, ld=c + 1, fill=rand(rng, r, c))
        db = torch.zeros(rows, dtype=F32, device=dev()) if bias else None
        old = w64(dw, layout)
        Z.zero_linear_grad_weight(dz.t, x.t, dw.t, db, w_layout=layout, accumulate=True)
        want, err = R.linear_grad_weight(dz.f64(), x.f64(), old=old, out="f32")
        close("dw", dw.t if layout == 0 else dw.t.t(), want, err)
        assert dw.intact_outside()
    want, err = R.column_sums(dz.f64(), out="f32")
    close("db", db, want, err)


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("inner", [264, 129, 1])
@pytest.mark.parametrize("odd", ["a", "b"])
def test_one_operand_of_odd_rows(Z, odd, inner, layout):
    """One operand with rows on 16 bytes, the other without, in each direction."""
    rng = rng_of((19, odd, inner, layout))
    say("one odd", odd, inner, layout)
    rows, cols = 301, 203

    def mat(which, r, c):
        return inp(rng, r, c, scale=0.3, pad_ld=-c % 8 + (5 if which == odd else 0), shift=3 if which == odd else 0)

    x, w = mat("a", rows, inner), mat("b", *((cols, inner) if layout == 0 else (inner, cols)))
    y = Mat(rows, cols, F32, ld=cols + 1)
    Z.zero_linear_forward(x.t, w.t, w_layout=layout, y=y.t)
    want, err, _, _ = R.linear_forward(x.f64(), w64(w, layout), out="f32")
    close("y", y.t, want, err)
    dz, w = mat("a", rows, inner), mat("b", *((inner, cols) if layout == 0 else (cols, inner)))
    dx = Mat(rows, cols, BF, ld=cols + 1)
    Z.zero_linear_grad_input(dz.t, w.t, w_layout=layout, dx=dx.t)
    want, err = R.linear_grad_input(dz.f64(), w64(w, layout))
    close("dx", dx.t, want, err)
    dz, x = mat("a" if layout == 0 else "b", inner, rows), mat("b" if layout == 0 else "a", inner, cols)
    r, c = (rows, cols) if layout == 0 else (cols, rows)
    dw, db = Mat(r, c, F32, ld=c + 3), torch.empty(rows, dtype=F32, device=dev())
    Z.zero_linear_grad_weight(dz.t, x.t, dw.t, db, w_layout=layout)
    want, err = R.linear_grad_weight(dz.f64(), x.f64(), out="f32")
    close("dw", dw.t if layout == 0 else dw.t.t(), want, err)
    want, err = R.column_sums(dz.f64(), out="f32")
    close("db", db, want, err)
    assert y.intact_outside() and dx.intact_outside() and dw.intact_outside()


@pytest.mark.parametrize("rows,cols", [(8190, 765), (8190, 2810), (5000, 4000), (3, 777)])
def test_empty_reduction(Z, rows, cols):
    """No inputs at all: the epilogue of zeros, in each kind of tile."""
    rng = rng_of((21, rows, cols))
    x, w = torch.empty((rows, 0), dtype=BF, device=dev()), torch.empty((cols, 0), dtype=BF, device=dev())
    res, b = inp(rng, rows, cols), inp(rng, 1, cols)
    y = Z.zero_linear_forward(x, w, b.t[0], residual=res.t, dtype=BF)
    assert torch.equal(y, (res.t.float() + b.t.float()).to(BF))
    dx = Z.zero_linear_grad_input(x, torch.empty((0, cols), dtype=BF, device=dev()), dtype=F32)
    assert torch.equal(dx, torch.zeros_like(dx))
    dw = torch.full((rows, cols), 3.5, dtype=BF, device=dev())
    dz, a = torch.empty((0, rows), dtype=BF, device=dev()), torch.empty((0, cols), dtype=BF, device=dev())
    Z.zero_linear_grad_weight(dz, a, dw, accumulate=True)
    assert bool((dw == 3.5).all())
    Z.zero_linear_grad_weight(dz, a, dw)
    assert not bool(dw.any())


def test_captured_calls_of_many_tiles(Z):
    """Products in one launch and in two, split reductions with their join and the bias
    gradient, captured on one workspace: every replay equals the eager calls, with eager
    work on a workspace of its own between replays."""
    rng = rng_of((22,))
    x, w, dy = inp(rng, 8190, 200), inp(rng, 765, 200, scale=0.1, pad_ld=0), inp(rng, 8190, 765, pad_ld=3)
    wide = inp(rng, 2810, 968, scale=0.03)
    h = inp(rng, 8190, 968)
    need = max(Z.zero_linear_workspace_bytes(k, 0, 8190, a, b) for k in range(3) for a, b in ((200, 765), (968, 2810)))
    assert need > 0

    def outs():
        z = lambda r, c, t: torch.zeros((r, c), dtype=t, device=dev())
        return (z(8190, 765, BF), z(8190, 200, BF), z(765, 200, F32), z(1, 765, F32)[0], z(8190, 2810, BF),
                torch.empty(need, dtype=torch.uint8, device=dev()))

    def calls(drop, y, dx, dw, db, v, ws):
        Z.zero_linear_forward(x.t, w.t, dropout=drop, y=y, workspace=ws)
        Z.zero_linear_grad_input(dy.t, w.t, dropout=drop, dx=dx, workspace=ws)
        Z.zero_linear_grad_weight(dy.t, x.t, dw, db, accumulate=True, workspace=ws)
        Z.zero_linear_forward(h.t, wide.t, act=3, dropout=drop, y=v, workspace=ws)

    counter = torch.zeros(1, dtype=torch.int64, device=dev())
    drop = Z.zero_dropout(0.25, 6, 1, counter=counter)
    got, want = outs(), outs()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(s):
        calls(drop, *got)
        torch.cuda.synchronize()
        got[2].zero_(), got[3].zero_()
        with torch.cuda.graph(graph, stream=s):
            calls(drop, *got)
    torch.cuda.synchronize()
    for k in range(4):
        counter.fill_(k)
        graph.replay()
        calls(Z.zero_dropout(0.25, 6, 1 + k), *want)
        torch.cuda.synchronize()
        for name, a, b in zip("y dx dw db v".split(), got, want):
            assert torch.equal(a, b), (k, name)


@pytest.mark.parametrize("N", [(1 << 26) - 3, (1 << 26) + 9])
def test_most_columns(Z, N):
    """Both sides of the width up to which one row takes a launch of its own."""
    g = torch.Generator(device=dev()).manual_seed(N)
    x = torch.randn((1, 1), dtype=BF, device=dev(), generator=g)
    w = torch.randn((N, 1), dtype=BF, device=dev(), generator=g)
    y = Z.zero_linear_forward(x, w)
    want = (x.float() * w.float()[:, 0]).to(BF)         # exact in f32, one rounding
    assert torch.equal(y, want)


def test_most_rows(Z):
    """A million tiles below one another."""
    M = (1 << 27) + 5
    g = torch.Generator(device=dev()).manual_seed(M)
    dz = torch.randn((M, 1), dtype=BF, device=dev(), generator=g)
    w = torch.randn((1, 1), dtype=BF, device=dev(), generator=g)
    dx = Z.zero_linear_grad_input(dz, w)
    assert torch.equal(dx, (dz.float() * w.float()).to(BF))


def test_dropout_of_more_than_one_launch(Z):
    """2^31 threads and more: the rows around the seam and the last ones are as those of
    a matrix that a call of few rows gives."""
    N = 8192
    M = (1 << 21) + 7                                   # 1024 threads a row
    if torch.cuda.mem_get_info()[0] < 3 * M * N:
        pytest.skip("not enough free memory")
    p, seed = 0.25, 11
    x = torch.empty((M, N), dtype=BF, device=dev())
    for r in (0, (1 << 21) - 2, (1 << 21) - 1, 1 << 21, M - 1):
        x[r].fill_(1.0)
    Z.zero_dropout_add(x, Z.zero_dropout(p, seed, 3), y=x)
    for r in (0, (1 << 21) - 2, (1 << 21) - 1, 1 << 21, M - 1):
        want = R.drop_row(r, N, p, seed, 3)
        got = x[r].float().cpu().numpy().astype(np.float64)
        assert (np.abs(got - want) <= 2.0 ** -8 * np.abs(want)).all(), r
