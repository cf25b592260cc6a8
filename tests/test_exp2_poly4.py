"""The serving softmax's polynomial 2^x on the CPU: coefficients against the fit that has the least
relative error, the error of its steps, exact powers of two, the clamp."""
import numpy as np
import pytest

from tests import exp2_poly4_ref as R


def test_coefficients_have_the_least_error():
    linprog = pytest.importorskip("scipy.optimize").linprog
    f = np.linspace(-0.5, 0.5, 4001)
    y, A, S = 2.0 ** f, np.stack([f ** k for k in (1, 2, 3, 4)], 1), 1e5
    # |1 + A c - y| <= (e / S) y, with e the objective (scaled: the error is near the solver's own)
    r = linprog([0, 0, 0, 0, 1], A_ub=np.vstack([np.hstack([A, -y[:, None] / S]), np.hstack([-A, -y[:, None] / S])]),
                b_ub=np.concatenate([y - 1.0, 1.0 - y]), bounds=[(None, None)] * 5, method="highs",
                options=dict(primal_feasibility_tolerance=1e-10, dual_feasibility_tolerance=1e-10))
    assert r.success, r.message
    c = np.array(R.constants(), dtype=np.float64)
    err = np.abs((1 + A @ c) / y - 1).max()
    # rounding the coefficients to 32 bits moves the value by at most sum 2^-25 c_k |f|^k / 2^f < 2^-25
    assert err <= r.x[4] / S + 2.0 ** -25 and err <= R.BOUND - 2.0 ** -23
    assert np.abs(c - r.x[:4]).max() < 1e-7


def test_error_powers_of_two_and_clamp():
    x = R.points()
    R.check(x, R.poly4(x))


def test_planted_mistakes_are_found(monkeypatch):
    x = R.points()
    c = R.constants()
    for i in range(4):
        bad = list(c)
        bad[i] = np.float32(bad[i] * (1 + 1e-3))
        monkeypatch.setattr(R, "constants", lambda bad=bad: bad)
        with pytest.raises(AssertionError):
            R.check(x, R.poly4(x))
