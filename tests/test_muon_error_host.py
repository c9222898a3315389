"""The allowance of tests/muon_error_ref.py (CPU only): it holds for a model of pairs of fp16
numbers and for fp32, and does not hold for fewer bits."""
import numpy as np
import pytest
import torch

import muon_error_ref as E
import muon_ref as R


def in_32_bits(x, steps):
    f = np.float32
    X = np.asarray(x, f) / f(np.sqrt((np.asarray(x, np.float64) ** 2).sum()) + 1e-7)
    tall = X.shape[0] > X.shape[1]
    X = X.T.copy() if tall else X
    a, b, c = (f(v) for v in R.COEF)
    for _ in range(steps):
        A = X @ X.T
        X = a * X + (b * A + c * (A @ A)) @ X
    return X.T if tall else X


def rounded(x):
    return torch.from_numpy(np.ascontiguousarray(x, np.float32)).to(torch.bfloat16).double().numpy()


@pytest.mark.parametrize("kind,rows,cols,steps", E.CASES)
def test_models_are_within_what_arithmetic_allows(kind, rows, cols, steps):
    x = E.matrix(kind, rows, cols, np.random.default_rng(rows * 1000 + cols))
    x = x.astype(np.float32).astype(np.float64)
    want, allowed = E.growth(x, steps=steps)
    pairs, singles = (np.linalg.norm(v - want) for v in (E.model(x, steps=steps), in_32_bits(x, steps)))
    assert pairs <= allowed and singles <= allowed
    assert pairs <= 4 * singles + 2.0 ** -22 * np.linalg.norm(want)         # as the header says
    assert pairs <= 2.0 ** -20 * R.COEF[0] ** steps * np.linalg.norm(want)
    assert E.beyond_rounding(rounded(E.model(x, steps=steps)), want) <= allowed


@pytest.mark.parametrize("kind,rows,cols,steps", [c for c in E.CASES if c[1] >= 64 and c[3] == 5])
def test_the_allowance_sees_fewer_bits(kind, rows, cols, steps):
    """fp16 operands and 18 bits of X leave more than is allowed, through o's rounding too where the
    matrix is of more than a few directions; so does a mistake in the formula."""
    x = E.matrix(kind, rows, cols, np.random.default_rng(rows * 1000 + cols))
    want, allowed = E.growth(x, steps=steps)
    if kind != "rank1":
        assert np.linalg.norm(R.model(x) - want) > allowed
    if kind not in ("rank1", "rank6"):
        assert E.beyond_rounding(rounded(R.model(x)), want) > allowed
    wrong = R.orthogonalize(x, steps=steps, coefficients=(3.4445, -4.7750, 2.0815))
    assert E.beyond_rounding(rounded(wrong), want) > allowed


def test_a_table_of_larger_gains():
    x = E.matrix("rank6", 200, 300, np.random.default_rng(4))
    want, allowed = E.growth(x, coefficients=E.TABLE)
    assert np.linalg.norm(E.model(x, coefficients=E.TABLE) - want) <= allowed


def test_steps_that_would_grow_roundings_are_refused():
    """The product of the a's above 1 is bounded, where there is nothing to do as well: seven steps
    of the default coefficients, twelve of a = 2, any number of a at most 1."""
    import ctypes

    import zero_partitioned_optimizer_amd as Z
    from zero_partitioned_optimizer_amd import _binding as B
    from zero_partitioned_optimizer_amd import muon as M

    def call(steps, triples=None, batch=0):
        flat = None if triples is None else [v for t in triples for v in t]
        a = Z.zero_orthogonalize_args(batch=batch, rows=4, cols=4, steps=steps, eps=1e-7, scale=1.0, x_dtype=B.ZERO_F32,
                                      ld_x=4, ld_o=4,
                                      coefficients=None if flat is None else (ctypes.c_double * len(flat))(*flat))
        return M._lib().zero_orthogonalize(a, None)

    for steps, triples in ((7, None), (13, [(2.0, -1.5, 0.5)] * 13), (5, E.TABLE), (64, [(1.0, -0.5, 0.0)] * 64),
                           (64, [(0.25, 0.0, 0.0)] * 63 + [(8192.0, 0.0, 0.0)])):
        assert call(steps, triples) == B.ZERO_OK
    for steps, triples in ((8, None), (64, None), (14, [(2.0, -1.5, 0.5)] * 14), (14, [(-2.0, 1.5, -0.5)] * 14),
                           (5, [E.TABLE[0]] * 5)):
        for batch in (0, 1):
            assert call(steps, triples, batch) == B.ZERO_E_INVAL and "multiply to" in Z.zero_last_error()
