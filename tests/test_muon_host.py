"""The matrix step's argument checks (synchronous, before any launch, so that they run
without a GPU), and the 64-bit reference and rounding model of the GPU tests."""
import ctypes

import numpy as np
import pytest
import torch

import muon_ref as R
import zero_partitioned_optimizer_amd as Z
from zero_partitioned_optimizer_amd import _binding as B
from zero_partitioned_optimizer_amd import muon as M

BASE = 1 << 40                      # addresses that nothing reads: every call here is refused
INVAL, ALIGN, RANGE = B.ZERO_E_INVAL, B.ZERO_E_ALIGN, B.ZERO_E_RANGE


def call(fn, a):
    return getattr(M._lib(), fn)(a, None)


def momentum_args(**kw):
    a = Z.zero_muon_momentum_args(n=64, grad=BASE, momentum=BASE + 0x1000, u=BASE + 0x2000, grad_dtype=B.ZERO_F32,
                                  u_dtype=B.ZERO_BF16, nesterov=1, mu=0.95)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def update_args(**kw):
    a = Z.zero_muon_update_args(n=64, p=BASE, o=BASE + 0x1000, slot_bf16=BASE + 0x2000, lr=0.02, weight_decay=0.1)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def orth_args(**kw):
    a = Z.zero_orthogonalize_args(batch=2, rows=12, cols=20, x=BASE, ld_x=20, stride_x=240, o=BASE + 0x10000, ld_o=20,
                                  stride_o=240, x_dtype=B.ZERO_BF16, steps=5, eps=1e-7, scale=1.0,
                                  workspace_dev=BASE + 0x100000, ws_bytes=1 << 30)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("kw,status,word", [
    (dict(n=-1), RANGE, "n=-1"),
    (dict(n=(1 << 40) + 1), RANGE, "2^40"),
    (dict(grad=None), INVAL, "grad is NULL"),
    (dict(momentum=None), INVAL, "momentum is NULL"),
    (dict(u=None), INVAL, "u is NULL"),
    (dict(grad=BASE + 2), ALIGN, "grad="),
    (dict(u=BASE + 0x2001), ALIGN, "u="),
    (dict(stats_dev=BASE + 0x5004), ALIGN, "stats_dev="),
    (dict(grad_dtype=B.ZERO_BF16_WIRE), INVAL, "grad_dtype"),
    (dict(u_dtype=5), INVAL, "u_dtype"),
    (dict(mu=1.0), INVAL, "mu=1"),
    (dict(mu=-0.1), INVAL, "mu="),
    (dict(mu=float("nan")), INVAL, "mu="),
    (dict(momentum=BASE), INVAL, "overlap"),
    (dict(u=BASE), INVAL, "overlap"),                       # of another type than grad
    (dict(u=BASE + 0x1000), INVAL, "overlap"),
    (dict(stats_dev=BASE + 0x2010), INVAL, "overlap"),
])
def test_momentum_refuses(kw, status, word):
    assert call("zero_muon_momentum", momentum_args(**kw)) == status
    assert word in Z.zero_last_error() and "zero_muon_momentum" in Z.zero_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(n=-1), RANGE, "n=-1"),
    (dict(p=None), INVAL, "p is NULL"),
    (dict(o=None), INVAL, "o is NULL"),
    (dict(p=BASE + 2), ALIGN, "p="),
    (dict(slot_bf16=BASE + 0x2001), ALIGN, "slot_bf16="),
    (dict(lr=-1.0), INVAL, "lr="),
    (dict(lr=float("inf")), INVAL, "lr="),
    (dict(weight_decay=float("nan")), INVAL, "weight_decay="),
    (dict(slot_bf16=BASE + 0x1000), INVAL, "overlap"),
    (dict(o=BASE + 4), INVAL, "overlap"),
])
def test_update_refuses(kw, status, word):
    assert call("zero_muon_update", update_args(**kw)) == status
    assert word in Z.zero_last_error() and "zero_muon_update" in Z.zero_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(batch=-1), RANGE, "-1 matrices"),
    (dict(batch=1 << 31), RANGE, "matrices"),
    (dict(rows=-1), RANGE, "-1 x 20"),
    (dict(rows=1 << 16, cols=1 << 16), RANGE, "smaller side"),
    (dict(rows=(1 << 20) + 1), RANGE, "larger"),
    (dict(steps=0), INVAL, "steps=0"),
    (dict(steps=65), INVAL, "steps=65"),
    (dict(x_dtype=B.ZERO_BF16_WIRE), INVAL, "x_dtype"),
    (dict(eps=0.0), INVAL, "eps="),
    (dict(eps=float("nan")), INVAL, "eps="),
    (dict(scale=float("inf")), INVAL, "scale="),
    (dict(scale=2e4), INVAL, "scale="),
    (dict(coefficients=(ctypes.c_double * 15)(*[1.0] * 14, float("nan"))), INVAL, "coefficient"),
    (dict(x=None), INVAL, "x is NULL"),
    (dict(o=None), INVAL, "o is NULL"),
    (dict(x=BASE + 1), ALIGN, "x="),
    (dict(x=BASE + 2, x_dtype=B.ZERO_F32), ALIGN, "x="),
    (dict(ld_x=19), RANGE, "ld of x"),
    (dict(ld_o=(1 << 40) + 1), RANGE, "ld of o"),
    (dict(stride_x=239), RANGE, "batch stride of x"),
    (dict(stride_o=0), RANGE, "batch stride of o"),
    (dict(stride_o=-240), RANGE, "batch stride of o"),
    (dict(stride_x=(1 << 50) + 1), RANGE, "batch stride of x"),
    (dict(batch=(1 << 31) - 1, stride_x=1 << 50), RANGE, "address space"),
    (dict(o=BASE), INVAL, "overlap"),
    (dict(o=BASE + 400), INVAL, "overlap"),
    (dict(workspace_dev=None), INVAL, "workspace_dev is NULL"),
    (dict(workspace_dev=BASE + 0x100004), ALIGN, "workspace_dev"),
    (dict(ws_bytes=1000), RANGE, "ws_bytes"),
    (dict(workspace_dev=BASE), INVAL, "overlap"),
])
def test_orthogonalize_refuses(kw, status, word):
    assert call("zero_orthogonalize", orth_args(**kw)) == status
    assert word in Z.zero_last_error() and "zero_orthogonalize" in Z.zero_last_error()


@pytest.mark.parametrize("fn", ["zero_muon_momentum", "zero_muon_update", "zero_orthogonalize"])
def test_null_args(fn):
    assert call(fn, None) == INVAL and "args is NULL" in Z.zero_last_error()


def test_nothing_to_do():
    assert call("zero_muon_momentum", momentum_args(n=0, grad=None)) == B.ZERO_OK
    assert call("zero_muon_update", update_args(n=0, p=None)) == B.ZERO_OK
    for size in (dict(batch=0), dict(rows=0), dict(cols=0)):
        assert call("zero_orthogonalize", orth_args(x=None, **size)) == B.ZERO_OK


def test_workspace():
    """Enough for one matrix of a group of at most 4 GiB, and no more for a longer stack."""
    need = Z.zero_orthogonalize_workspace_bytes
    assert need(0, 8, 8) == need(1, 0, 8) == need(-1, 8, 8) == need(1, 1 << 16, 1 << 16) == 0
    one = need(1, 768, 2304)
    assert one >= 768 * 2304 * 5 + 768 * 768 * 4 and need(12, 768, 2304) == 12 * one
    assert need(1, 2304, 768) == one
    most = need(100000, 768, 2304)
    assert most <= 4 << 30 and most == need(200000, 768, 2304) and most % one == 0
    assert need(3, 1 << 15, 1 << 20) == need(1, 1 << 15, 1 << 20) > 4 << 30


def test_binding_refuses():
    x = torch.zeros(4, 8, dtype=torch.bfloat16)
    for f in (lambda: Z.zero_orthogonalize(x), lambda: Z.zero_muon_momentum(x[0], x[0].float()),
              lambda: Z.zero_muon_update(x[0].float(), x[0], lr=0.1)):
        with pytest.raises(Z.ZeroError, match="not on the current device"):
            f()
    for bad in ((1.0, 2.0), [(1.0, 2.0, 3.0)] * 4, (1.0, 2.0, 3.0, 4.0)):
        with pytest.raises(Z.ZeroError, match="neither three numbers nor 5 triples"):
            M._table(M._coefficients(bad), 5)
    assert list(M._table(M._coefficients([(1, 2, 3), (4, 5, 6)]), 2)) == [1, 2, 3, 4, 5, 6]
    assert list(M._table(M._coefficients(np.arange(1, 7).reshape(2, 3)), 2)) == [1, 2, 3, 4, 5, 6]
    assert list(M._table(R.COEF, 2)) == list(R.COEF) * 2


def matrix(kind, R_, C):
    rng = np.random.default_rng(R_ * 1000 + C)
    if kind == "rank1":
        x = rng.standard_normal((R_, 1)) * rng.standard_normal((1, C))
    elif kind == "rank4":
        x = rng.standard_normal((R_, 4)) @ rng.standard_normal((4, C))
    else:
        x = rng.standard_normal((R_, C))
    return torch.from_numpy(x).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("kind", ["normal", "rank1", "rank4"])
@pytest.mark.parametrize("size", [(1, 1), (1, 50), (50, 1), (8, 8), (40, 40), (30, 90), (90, 30), (16, 700), (257, 120), (512, 512)])
def test_rounding_model_is_near_the_formula(kind, size):
    """The documented precision: 2e-3 of the result's norm before o is rounded, 4e-3 where a side
    is below 32, whatever the fall of the singular values; and the formula's singular values
    are near 1."""
    x = matrix(kind, *size)
    want = R.orthogonalize(x)
    assert np.linalg.norm(R.model(x) - want) <= (2e-3 if min(size) >= 32 else 4e-3) * np.linalg.norm(want)
    s = np.linalg.svd(want, compute_uv=False)
    rank = {"rank1": 1, "rank4": min(4, *size), "normal": 1}[kind]
    assert s.max() < 1.3 and s[rank - 1] > 0.6
    assert np.allclose(R.orthogonalize(x.T), want.T, atol=1e-12)


def test_the_bounds_see_mistakes():
    """A planted mistake in the formula is far outside what the GPU tests allow."""
    x = matrix("normal", 60, 100)
    want, each, whole = R.bounds(x)
    for kw in (dict(steps=4), dict(coefficients=(3.4445, -4.7750, 2.0415)), dict(scale=1.02), dict(eps=1.0)):
        off = R.orthogonalize(x, **kw) - want
        assert np.linalg.norm(off) > whole and (np.abs(off) > each).any(), kw
    wrong = want.copy()
    wrong[3, 5] = -wrong[3, 5]
    assert (np.abs(wrong - want) > each).any()


def test_matrix_step_stacks_and_refusals():
    """Runs of one shape at even distances, and the layouts that are refused before any GPU work."""
    S = Z.MuonShardStep._stacks
    assert S([(0, 2, 3), (6, 2, 3), (12, 2, 3), (20, 3, 2), (30, 2, 3)]) == [(3, 0, 6, 2, 3), (1, 30, 6, 2, 3),
                                                                             (1, 20, 6, 3, 2)]
    assert S([(4, 2, 3), (14, 2, 3)]) == [(2, 4, 10, 2, 3)] and S([]) == []
    p0 = torch.zeros(100)
    for matrices, text in (([(0, 5, 10), (49, 5, 10)], "overlap"), ([(60, 1, 1), (59, 2, 1)], "overlap"),
                           ([(-1, 5, 10)], "matrix at -1")):
        with pytest.raises(Z.ZeroError, match=text):
            Z.MuonShardStep(100, 1, Z.ZERO_F32, p0, matrices, lr=0.1)
    with pytest.raises(Z.ZeroError, match="p0"):
        Z.MuonShardStep(100, 1, Z.ZERO_F32, p0, [(0, 5, 10)], lr=0.1)
