"""The 64-bit oracle of the operators around the layer, pinned by central
differences of its own forward functions: every gradient formula the GPU tests
compare with."""
import numpy as np
import pytest

from oracle import block as O


def _diff(f, v, i, eps=1e-5):
    a, b = v.copy(), v.copy()
    a[i] += eps
    b[i] -= eps
    return (f(a) - f(b)) / (2 * eps)


def test_rmsnorm_backward_against_differences():
    rng = np.random.default_rng(0)
    h, w, dy = rng.normal(size=(3, 256)), 1 + 0.1 * rng.normal(size=256), rng.normal(size=(3, 256))
    dres = rng.normal(size=(3, 256))
    eps = 1e-2
    _, rstd = O.rmsnorm(h, w, eps)
    dx, dw = O.rmsnorm_backward(dy, h, rstd, w, dres)
    f = lambda v: (O.rmsnorm(v, w, eps)[0] * dy).sum() + (v * dres).sum()  # noqa: E731
    g = lambda v: (O.rmsnorm(h, v, eps)[0] * dy).sum()  # noqa: E731
    for i in [(0, 0), (1, 17), (2, 255), (2, 128)]:
        assert abs(_diff(f, h, i) - dx[i]) <= 1e-7 * max(1, abs(dx[i]))
    for i in [0, 100, 255]:
        assert abs(_diff(g, w, i) - dw[i]) <= 1e-7 * max(1, abs(dw[i]))


@pytest.mark.parametrize("Nr,Kr,off", [(16, 4, [0, 5, 5, 12]), (7, 1, [2, 3, 9])])
def test_balance_and_gates_against_differences(Nr, Kr, off):
    rng = np.random.default_rng(Nr)
    T = 12
    z = rng.normal(size=(T, Nr)) * 1.7
    idx = np.argsort(-z, axis=1)[:, :Kr]
    dloss = rng.normal(size=len(off) - 1)
    dgate = rng.normal(size=(T, Kr))
    rs = 2.5
    loss, counts = O.balance_loss(z, idx, off, 0.3)
    assert counts.sum() == (off[-1] - off[0]) * Kr
    assert loss[np.diff(off) == 0].sum() == 0

    def f(v):
        s, _ = O.sigmoid(v)
        sel = np.take_along_axis(s, idx, axis=1)
        gate = rs * sel / sel.sum(axis=1, keepdims=True)
        return (O.balance_loss(v, idx, off, 0.3)[0] * dloss).sum() + (gate * dgate).sum()

    dz, mag = O.router_dlogits(z, idx, dgate=dgate, route_scale=rs, off=off, counts=counts, dloss=dloss, alpha=0.3)
    for i in [(0, 0), (2, 3), (5, 6), (11, 1), (4, int(idx[4, 0]))]:
        assert abs(_diff(f, z, i) - dz[i]) <= 1e-8
    assert (mag + 1e-15 >= np.abs(dz)).all()


def test_sigmoid_keeps_the_small_side():
    s, om = O.sigmoid(np.array([40.0, -40.0, 0.0]))
    assert om[0] == pytest.approx(np.exp(-40.0), rel=1e-12) and s[1] == pytest.approx(np.exp(-40.0), rel=1e-12)
    assert s[2] == om[2] == 0.5
