"""The layer operators' argument checks (synchronous, before any launch, so that they
run without a GPU), and the 64-bit reference that the GPU tests use: the generator
against its published test vectors, slopes against differences."""
import ctypes

import numpy as np
import pytest
import torch  # noqa: F401

import layer_ref as R
import zero_partitioned_optimizer_amd as Z
from zero_partitioned_optimizer_amd import _binding as B
from zero_partitioned_optimizer_amd import layer as L

BASE = 1 << 40                      # addresses that nothing reads: every call here is refused


def call(fn, a):
    return getattr(L._lib(), fn)(a, None)


def forward_args(**kw):
    a = Z.zero_linear_args(M=4, K=16, N=24, x=BASE, ld_x=16, w=BASE + 0x10000, ld_w=16, w_layout=0, act=0,
                           y=BASE + 0x20000, ld_y=24, y_dtype=B.ZERO_BF16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def grad_input_args(**kw):
    a = Z.zero_linear_grad_input_args(M=4, K=16, N=24, dz=BASE, ld_dz=24, w=BASE + 0x10000, ld_w=16, w_layout=0,
                                      act=0, dx=BASE + 0x20000, ld_dx=16, dx_dtype=B.ZERO_BF16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def grad_weight_args(**kw):
    a = Z.zero_linear_grad_weight_args(M=4, K=16, N=24, dz=BASE, ld_dz=24, x=BASE + 0x10000, ld_x=16,
                                       dw=BASE + 0x20000, ld_dw=16, w_layout=0, grad_dtype=B.ZERO_BF16,
                                       workspace_dev=BASE + 0x100000, ws_bytes=1 << 26)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


def dropout_args(**kw):
    a = Z.zero_dropout_args(M=4, N=24, x=BASE, ld_x=24, y=BASE + 0x20000, ld_y=24, x_dtype=B.ZERO_BF16,
                            y_dtype=B.ZERO_BF16)
    for k, v in kw.items():
        setattr(a, k, v)
    return a


INVAL, ALIGN, RANGE = B.ZERO_E_INVAL, B.ZERO_E_ALIGN, B.ZERO_E_RANGE


@pytest.mark.parametrize("kw,status,word", [
    (dict(M=-1), RANGE, "M=-1"),
    (dict(N=1 << 31), RANGE, "N="),
    (dict(M=(1 << 29) + 1), RANGE, "2^29 a side"),
    (dict(M=1 << 20, N=1 << 18, ld_w=1 << 18, ld_y=1 << 18), RANGE, "2^23 tiles"),
    (dict(x=None), INVAL, "x is NULL"),
    (dict(w=None), INVAL, "w is NULL"),
    (dict(y=None), INVAL, "y is NULL"),
    (dict(x=BASE + 1), ALIGN, "x="),
    (dict(y=BASE + 0x20002, y_dtype=B.ZERO_F32), ALIGN, "y="),
    (dict(ld_x=15), RANGE, "ld of x"),
    (dict(ld_w=15), RANGE, "ld of w"),
    (dict(w_layout=1, ld_w=23), RANGE, "ld of w"),
    (dict(ld_y=(1 << 40) + 1), RANGE, "ld of y"),
    (dict(w_layout=2), INVAL, "w_layout"),
    (dict(act=4), INVAL, "act"),
    (dict(act=-1), INVAL, "act"),
    (dict(y_dtype=B.ZERO_BF16_WIRE), INVAL, "y_dtype"),
    (dict(dropout=Z.zero_dropout(1.0)), INVAL, "dropout"),
    (dict(dropout=Z.zero_dropout(-0.1)), INVAL, "dropout"),
    (dict(dropout=Z.zero_dropout(float("nan"))), INVAL, "dropout"),
    (dict(y=BASE), INVAL, "overlap"),
    (dict(y=BASE + 0x10000 + 2), INVAL, "overlap"),
    (dict(preact=BASE + 0x20000, ld_preact=24), INVAL, "overlap"),
    (dict(preact=BASE + 0x20000 + 16, ld_preact=24), INVAL, "overlap"),
    (dict(residual=BASE + 0x20002, ld_residual=24), INVAL, "overlap"),
    (dict(residual=BASE + 0x20000, ld_residual=32), INVAL, "overlap"),
    (dict(bias=BASE + 0x20010), INVAL, "overlap"),
])
def test_forward_refuses(kw, status, word):
    assert call("zero_linear_forward", forward_args(**kw)) == status
    assert word in Z.zero_last_error() and "zero_linear_forward" in Z.zero_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(K=-5), RANGE, "K=-5"),
    (dict(dz=None), INVAL, "dz is NULL"),
    (dict(dx=None), INVAL, "dx is NULL"),
    (dict(act=1), INVAL, "preact is NULL"),
    (dict(act=1, preact=BASE + 0x30001, ld_preact=16), ALIGN, "preact"),
    (dict(act=1, preact=BASE + 0x30000, ld_preact=8), RANGE, "ld of preact"),
    (dict(act=2, preact=BASE + 0x20000, ld_preact=24), INVAL, "overlap"),
    (dict(act=2, preact=BASE + 0x20000, ld_preact=16, dx_dtype=B.ZERO_F32), INVAL, "overlap"),
    (dict(dx=BASE), INVAL, "overlap"),
    (dict(dx_dtype=7), INVAL, "dx_dtype"),
    (dict(dropout=Z.zero_dropout(2.0)), INVAL, "dropout"),
])
def test_grad_input_refuses(kw, status, word):
    assert call("zero_linear_grad_input", grad_input_args(**kw)) == status
    assert word in Z.zero_last_error()


@pytest.mark.parametrize("kw,status,word", [
    (dict(M=1 << 31), RANGE, "M="),
    (dict(dw=None), INVAL, "dw is NULL"),
    (dict(x=None), INVAL, "x is NULL"),
    (dict(dw=BASE + 0x20001), ALIGN, "dw="),
    (dict(dw=BASE + 0x20002, grad_dtype=B.ZERO_F32), ALIGN, "dw="),
    (dict(dbias=BASE + 0x20000 + 2 * 16 * 23), INVAL, "overlap"),
    (dict(dw=BASE), INVAL, "overlap"),
    (dict(ld_dw=15), RANGE, "ld of dw"),
    (dict(w_layout=1, ld_dw=16), RANGE, "ld of dw"),
    (dict(grad_dtype=2), INVAL, "grad_dtype"),
    (dict(workspace_dev=None), INVAL, "workspace_dev is NULL"),
    (dict(workspace_dev=BASE + 0x100008), ALIGN, "workspace_dev"),
    (dict(ws_bytes=3), RANGE, "ws_bytes"),
    (dict(workspace_dev=BASE + 0x10000), INVAL, "overlap"),
])
def test_grad_weight_refuses(kw, status, word):
    kw = dict({"dbias": BASE + 0x40000}, **kw)      # a bias gradient always needs the workspace
    assert call("zero_linear_grad_weight", grad_weight_args(**kw)) == status
    assert word in Z.zero_last_error()


@pytest.mark.parametrize("fn,kw,status,word", [
    ("zero_dropout_add", dict(M=-1), RANGE, "M=-1"),
    ("zero_dropout_add", dict(x=None), INVAL, "x is NULL"),
    ("zero_dropout_add", dict(y=BASE + 2), INVAL, "overlap"),
    ("zero_dropout_add", dict(y=BASE, y_dtype=B.ZERO_F32), INVAL, "overlap"),
    ("zero_dropout_add", dict(act=1), INVAL, "takes no act"),
    ("zero_dropout_add", dict(preact=BASE + 0x50000), INVAL, "takes no act"),
    ("zero_dropout_add", dict(x_dtype=3), INVAL, "x_dtype"),
    ("zero_dropout_add", dict(dropout=Z.zero_dropout(1 - 2.0 ** -17)), INVAL, "dropout"),
    ("zero_dropout_grad", dict(residual=BASE + 0x50000, ld_residual=24), INVAL, "residual"),
    ("zero_dropout_grad", dict(act=3), INVAL, "preact is NULL"),
    ("zero_dropout_grad", dict(act=9), INVAL, "act"),
    ("zero_dropout_grad", dict(x=BASE + 1), ALIGN, "dy="),
])
def test_dropout_refuses(fn, kw, status, word):
    assert call(fn, dropout_args(**kw)) == status
    assert word in Z.zero_last_error()


def test_null_args():
    for fn in ("zero_linear_forward", "zero_linear_grad_input", "zero_linear_grad_weight", "zero_dropout_add",
               "zero_dropout_grad"):
        assert call(fn, None) == INVAL


def test_counter_alignment():
    d = Z.zero_dropout(0.5)
    d.counter_dev = BASE + 4
    assert call("zero_dropout_add", dropout_args(dropout=d)) == ALIGN


def test_empty_calls_are_no_ops():
    """Nothing to write: no pointer is needed and nothing is launched."""
    for M, N in ((0, 8), (8, 0), (0, 0)):
        assert call("zero_linear_forward", Z.zero_linear_args(M=M, K=8, N=N)) == B.ZERO_OK
        assert call("zero_linear_grad_input", Z.zero_linear_grad_input_args(M=M, K=N, N=8)) == B.ZERO_OK
        assert call("zero_dropout_add", Z.zero_dropout_args(M=M, N=N)) == B.ZERO_OK
        assert call("zero_dropout_grad", Z.zero_dropout_args(M=M, N=N)) == B.ZERO_OK
    assert call("zero_linear_grad_weight", Z.zero_linear_grad_weight_args(M=8, K=8, N=0)) == B.ZERO_OK


def test_column_slices_of_one_buffer_do_not_overlap():
    """x and y as columns of the same rows are refused only where their columns meet:
    the adjacent ones pass the overlap check and are stopped by the unknown type
    that is checked before, or by the workspace after."""
    a = grad_weight_args(dz=BASE, ld_dz=64, x=BASE + 2 * 24, ld_x=64, dw=BASE + 2 * 40, ld_dw=64, ws_bytes=0,
                         workspace_dev=BASE + 0x100000, dbias=BASE + 0x40000)
    assert call("zero_linear_grad_weight", a) == RANGE and "ws_bytes" in Z.zero_last_error()
    a.dw = BASE + 2 * 39
    assert call("zero_linear_grad_weight", a) == INVAL and "overlap" in Z.zero_last_error()
    a.dw = BASE + 2 * 49                              # its rows wrap into the next row's dz
    assert call("zero_linear_grad_weight", a) == INVAL and "overlap" in Z.zero_last_error()


def test_workspace_bytes():
    assert Z.zero_linear_workspace_bytes(0, 0, -1, 8, 8) == 0
    assert Z.zero_linear_workspace_bytes(5, 0, 8, 8, 8) == 0
    assert Z.zero_linear_workspace_bytes(0, 2, 8, 4096, 8) == 0
    assert Z.zero_linear_workspace_bytes(0, 0, 0, 8, 8) == 0
    for kind in range(3):
        for M, K, N in ((1, 768, 2304), (8192, 768, 768), (8192, 4096, 11008), (1, 1, 1), (7, 50257, 3)):
            for layout in range(2):
                assert 0 <= Z.zero_linear_workspace_bytes(kind, layout, M, K, N) < 1 << 28
    with pytest.raises(Z.ZeroError):
        Z.zero_linear_forward(torch.zeros(2, 4), torch.zeros(3, 4))             # f32, on the CPU
    with pytest.raises(Z.ZeroError):
        Z.zero_linear_forward(torch.zeros(2, 4, dtype=torch.bfloat16), torch.zeros(3, 4, dtype=torch.bfloat16))


def test_struct_sizes_match_the_header():
    for s, n in ((Z.zero_linear_args, 176), (Z.zero_linear_grad_input_args, 152),
                 (Z.zero_linear_grad_weight_args, 112), (Z.zero_dropout_args, 128)):
        assert ctypes.sizeof(s) == n, (s, ctypes.sizeof(s))


# ---------------------------------------------------------------------------
# the reference itself
# ---------------------------------------------------------------------------


@pytest.mark.parametrize("counter,key,want", [
    ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
    ((0xFFFFFFFF,) * 4, (0xFFFFFFFF,) * 2, (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
    ((0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344), (0xA4093822, 0x299F31D0),
     (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1)),
])
def test_generator_known_answers(counter, key, want):
    """The published test vectors of Philox4x32-10."""
    got = R.philox([np.array([c], dtype=np.uint64) for c in counter], key)
    assert tuple(int(x[0]) for x in got) == want


def test_drop_rate_and_scale():
    f = R.drop_factor(512, 1003, 0.25, 99, 3)
    kept = (f != 0).mean()
    # 5 standard deviations of a mean of 512 * 1003 draws of probability 3/4
    assert abs(kept - 0.75) < 5 * np.sqrt(0.75 * 0.25 / f.size)
    assert set(np.unique(f)) == {0.0, 65536.0 / (65536 - 16384)}
    assert not np.array_equal(f, R.drop_factor(512, 1003, 0.25, 99, 4))
    assert not np.array_equal(f, R.drop_factor(512, 1003, 0.25, 100, 3))
    # rows and columns draw independently of the matrix's size
    assert np.array_equal(f[:7, :40], R.drop_factor(7, 40, 0.25, 99, 3))


@pytest.mark.parametrize("name", R.ACTS)
def test_slopes_against_differences(name):
    z = np.linspace(-6.013, 6.017, 401)
    h = 1e-5
    d = (R.act(name, z + h) - R.act(name, z - h)) / (2 * h)
    # a central difference is off by h^2/6 |act'''| (below 3 for these) plus rounding
    assert np.max(np.abs(d - R.slope(name, z))) < 1e-9 + 3 * h * h / 6 + 1e-16 * 12 / h
