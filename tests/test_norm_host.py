"""The norms' argument checks (synchronous, before any launch, so that they run without a
GPU), and the 64-bit reference of the GPU tests against differences and torch's own."""
import numpy as np
import pytest
import torch

import norm_ref as R
import zero_partitioned_optimizer_amd as Z
from zero_partitioned_optimizer_amd import _binding as B
from zero_partitioned_optimizer_amd import layer as L

BASE = 1 << 40                      # addresses that nothing reads: every call here is refused
INVAL, ALIGN, RANGE = B.ZERO_E_INVAL, B.ZERO_E_ALIGN, B.ZERO_E_RANGE
BF16, F32 = B.ZERO_BF16, B.ZERO_F32


def call(fn, a):
    return getattr(L._lib(), fn)(a, None)


def forward_args(**kw):
    a = Z.zero_norm_args(M=4, N=24, x=BASE, ld_x=24, weight=BASE + 0x8000, y=BASE + 0x20000, ld_y=24, x_dtype=BF16,
                         sum_dtype=BF16, y_dtype=BF16, eps=1e-5)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def grad_args(**kw):
    a = Z.zero_norm_grad_args(M=4, N=24, dy=BASE, ld_dy=24, x=BASE + 0x10000, ld_x=24, weight=BASE + 0x8000,
                              stats=BASE + 0x9000, dx=BASE + 0x20000, ld_dx=24, dweight=BASE + 0x30000,
                              dy_dtype=BF16, x_dtype=BF16, dx_dtype=BF16, grad_dtype=BF16,
                              workspace_dev=BASE + 0x100000, ws_bytes=1 << 26)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


SUM = dict(residual=BASE + 0x40000, ld_residual=24, sum=BASE + 0x50000, ld_sum=24)


@pytest.mark.parametrize("kw,status,word", [
    (dict(M=-1), RANGE, "M=-1"),
    (dict(M=1 << 31), RANGE, "M="),
    (dict(N=(1 << 24) + 1), RANGE, "2^24"),
    (dict(kind=2), INVAL, "kind 2"),
    (dict(kind=-1), INVAL, "kind"),
    (dict(x_dtype=B.ZERO_BF16_WIRE), INVAL, "x_dtype"),
    (dict(sum_dtype=7), INVAL, "sum_dtype"),
    (dict(y_dtype=-1), INVAL, "y_dtype"),
    (dict(eps=-1e-9), INVAL, "eps"),
    (dict(eps=float("nan")), INVAL, "eps"),
    (dict(eps=float("inf")), INVAL, "eps"),
    (dict(x=None), INVAL, "x is NULL"),
    (dict(y=None), INVAL, "y is NULL"),
    (dict(x=BASE + 1), ALIGN, "x="),
    (dict(y=BASE + 0x20002, y_dtype=F32), ALIGN, "y="),
    (dict(stats=BASE + 0x60002), ALIGN, "stats="),
    (dict(ld_x=23), RANGE, "ld of x"),
    (dict(ld_y=(1 << 40) + 1), RANGE, "ld of y"),
    (dict(residual=BASE + 0x40000, ld_residual=24), INVAL, "without a sum"),
    (dict(sum=BASE + 0x40000, ld_sum=24), INVAL, "without a residual"),
    (dict(SUM, ld_sum=20), RANGE, "ld of sum"),
    (dict(SUM, sum=BASE + 0x20000), INVAL, "overlap"),          # y and sum
    (dict(SUM, sum=BASE + 0x40002), INVAL, "overlap"),
    (dict(SUM, sum=BASE + 0x40000, ld_sum=32), INVAL, "overlap"),
    (dict(y=BASE, y_dtype=F32), INVAL, "overlap"),              # of another type than x
    (dict(y=BASE + 2), INVAL, "overlap"),
    (dict(bias=BASE + 0x20010), INVAL, "overlap"),
    (dict(stats=BASE + 0x20010), INVAL, "overlap"),
    (dict(stats=BASE + 0x10), INVAL, "overlap"),
])
def test_forward_refuses(kw, status, word):
    assert call("zero_norm_forward", forward_args(**kw)) == status
    assert word in Z.zero_last_error() and "zero_norm_forward" in Z.zero_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(N=-5), RANGE, "N=-5"),
    (dict(kind=3), INVAL, "kind"),
    (dict(dy_dtype=9), INVAL, "dy_dtype"),
    (dict(x_dtype=9), INVAL, "x_dtype"),
    (dict(dx_dtype=9), INVAL, "dx_dtype"),
    (dict(grad_dtype=B.ZERO_BF16_WIRE), INVAL, "grad_dtype"),
    (dict(dy=None), INVAL, "dy is NULL"),
    (dict(stats=None), INVAL, "stats is NULL"),
    (dict(dx=None), INVAL, "dx is NULL"),
    (dict(dweight=BASE + 0x30002, grad_dtype=F32), ALIGN, "dweight="),
    (dict(ld_dx=23), RANGE, "ld of dx"),
    (dict(residual_grad=BASE + 0x20002, ld_residual_grad=24), INVAL, "overlap"),
    (dict(dbias=BASE + 0x30000), INVAL, "overlap"),
    (dict(dweight=BASE), INVAL, "overlap"),
    (dict(dx=BASE + 0x9000), INVAL, "overlap"),
    (dict(workspace_dev=None), INVAL, "workspace_dev is NULL"),
    (dict(workspace_dev=BASE + 0x100008), ALIGN, "workspace_dev"),
    (dict(ws_bytes=16), RANGE, "ws_bytes"),
    (dict(workspace_dev=BASE + 0x20000), INVAL, "overlap"),
])
def test_grad_refuses(kw, status, word):
    assert call("zero_norm_grad", grad_args(**kw)) == status
    assert word in Z.zero_last_error() and "zero_norm_grad" in Z.zero_last_error()


@pytest.mark.parametrize("fn", ["zero_norm_forward", "zero_norm_grad"])
def test_null_args(fn):
    assert call(fn, None) == INVAL and "args is NULL" in Z.zero_last_error()


def test_nothing_to_do():
    assert call("zero_norm_forward", forward_args(M=0, x=None, y=None)) == B.ZERO_OK
    assert call("zero_norm_forward", forward_args(N=0, x=None, y=None)) == B.ZERO_OK
    assert call("zero_norm_grad", grad_args(N=0, dweight=None)) == B.ZERO_OK
    assert call("zero_norm_grad", grad_args(M=0, dweight=None)) == B.ZERO_OK


def test_workspace():
    assert Z.zero_norm_workspace_bytes(0, 24) == 0
    assert Z.zero_norm_workspace_bytes(1, 24) > 0
    for bad in ((-1, 24), (4, 0), (4, (1 << 24) + 1), (1 << 31, 4)):
        assert Z.zero_norm_workspace_bytes(*bad) == 0


def test_binding_refuses_host_tensors():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    with pytest.raises(Z.ZeroError, match="not on the current device"):
        Z.zero_norm_forward(x)
    with pytest.raises(Z.ZeroError, match="not on the current device"):
        Z.zero_norm_grad(x, x, None, torch.zeros(4, 2))


def test_flat_norm_refuses():
    with pytest.raises(Z.ZeroError, match="holds 9 elements"):
        Z.FlatNorm([0, 8], [8, 9], 0, 1, 8)
    with pytest.raises(Z.ZeroError, match="kind"):
        Z.FlatNorm([0], [8], 0, None, 8, kind=5)
    n = Z.FlatNorm([0, 8], [8, 8], 0, 1, 8)
    with pytest.raises(Z.ZeroError, match="does not hold"):
        n.use(torch.zeros(15, dtype=torch.bfloat16))
    with pytest.raises(Z.ZeroError, match="fetch or use first"):
        n.forward(torch.zeros(4, 8, dtype=torch.bfloat16))


@pytest.mark.parametrize("rms", [False, True])
def test_reference_against_differences_and_torch(rms):
    """The reference's gradient is that of its forward pass, and both are torch's."""
    rng = np.random.default_rng(5)
    M, N, eps = 3, 7, 1e-3
    x, w, b, dy = rng.standard_normal((M, N)), rng.standard_normal(N), rng.standard_normal(N), rng.standard_normal((M, N))

    def loss(x, w, b):
        return (dy * R.forward(x, w, b, rms=rms, eps=eps, out="f32")[0]).sum()

    stats = R.forward(x, w, b, rms=rms, eps=eps, out="f32")[2]
    (dx, _), (dw, _), (db, _) = R.grad(dy, x, w, stats, rms=rms, out="f32")
    h = 1e-6
    for got, which in ((dx, 0), (dw, 1), (db, 2)):
        args = [x, w, b]
        for i in np.ndindex(got.shape):
            up, down = [a.copy() for a in args], [a.copy() for a in args]
            up[which][i] += h
            down[which][i] -= h
            assert abs((loss(*up) - loss(*down)) / (2 * h) - got[i]) < 1e-7
    t = [torch.tensor(a, requires_grad=True) for a in (x, w, b)]
    y = torch.nn.functional.rms_norm(t[0], (N,), t[1], eps) + t[2] if rms else \
        torch.nn.functional.layer_norm(t[0], (N,), t[1], t[2], eps)
    assert np.allclose(y.detach().numpy(), R.forward(x, w, b, rms=rms, eps=eps, out="f32")[0], atol=1e-12)
    y.backward(torch.tensor(dy))
    for got, want in zip((dx, dw, db), t):
        assert np.allclose(got, want.grad.numpy(), atol=1e-11)
