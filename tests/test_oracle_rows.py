"""The fp64 definitions of the router, the row sort, the weighted sum and the
adapters, pinned on the CPU: small hand-computed values, and the gradients
against central differences of the forward definition.

Central differences with step h = 1e-5 of a function with third derivatives
of order 1 are off by h^2 / 6 plus rounding 1e-16 / h, about 3e-11; 1e-7
leaves room for larger derivatives."""
import numpy as np
import pytest

from oracle import rows


def test_route_by_hand():
    z = np.array([[0.0, np.log(2.0), np.log(5.0), -np.inf]])
    ids, w, c, loss, slope = rows.route(z, 2, renormalize=False, balance=1.0)
    assert ids.tolist() == [[2, 1]] and c.tolist() == [0, 1, 1, 0]
    assert np.allclose(w, [[5 / 8, 2 / 8]], rtol=1e-14)
    # E/(k n^2) sum_e c_e share_e = 4/2 * (2/8 + 5/8)
    assert np.isclose(loss, 2 * 7 / 8) and np.allclose(slope, [0, 2, 2, 0])
    _, w, _, _, _ = rows.route(z, 2, renormalize=True, scale=3.0)
    assert np.allclose(w, [[15 / 7, 6 / 7]])


def test_route_ties_and_rows_that_choose_nothing():
    z = np.array([[1.0, 1.0, 1.0], [-np.inf, -np.inf, -np.inf], [-np.inf, 2.0, -np.inf], [9.0, np.nan, 9.0]])
    ids, w, c, _, _ = rows.route(z, 2, mask=[True, True, True, False])
    assert ids.tolist() == [[0, 1], [-1, -1], [1, -1], [-1, -1]]
    assert np.allclose(w, [[.5, .5], [0, 0], [1, 0], [0, 0]]) and c.tolist() == [1, 2, 0]


def test_a_perfectly_even_router_has_loss_balance():
    """Every expert equally often with equal shares: E/(k n^2) * E * (k n / E) * (n / E) = 1."""
    E, n = 8, 16
    z = np.zeros((n, E))
    z[np.arange(n), np.arange(n) % E] = 1e-9
    assert np.isclose(rows.route(z, 1, balance=0.25)[3], 0.25)


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renorm", [True, False])
def test_route_gradient_against_differences(scoring, renorm):
    g = np.random.default_rng(5)
    T, E, k, scale = 6, 9, 3, 2.5
    z = g.standard_normal((T, E)) * 2
    z[1, 4] = -np.inf
    mask = np.array([True] * 5 + [False])
    dw, dl = g.standard_normal((T, k)), 0.7
    ids, _, counts, _, slope = rows.route(z, k, scoring, renorm, scale, 0.3, mask)

    def value(zz):
        i, w, c, loss, _ = rows.route(zz, k, scoring, renorm, scale, 0.3, mask)
        assert (i == ids).all()
        return (w * dw).sum() + dl * loss

    d = rows.route_backward(z, ids, dw, slope, dl, scoring, renorm, scale)
    h = 1e-5
    for t in range(T):
        for e in range(E):
            if np.isinf(z[t, e]):
                assert d[t, e] == 0
                continue
            up, dn = z.copy(), z.copy()
            up[t, e] += h
            dn[t, e] -= h
            assert abs((value(up) - value(dn)) / (2 * h) - d[t, e]) < 1e-7


def test_group_rows_by_hand():
    offsets, order, slot = rows.group_rows(np.array([[2, 0], [-1, 2], [0, 7]]), 3)
    assert offsets.tolist() == [0, 2, 2, 4]
    assert order.tolist() == [1, 4, 0, 3, 2, 5]
    assert slot.tolist() == [[2, 0], [-1, 3], [1, -1]]


def test_combine_gradient_against_differences():
    g = np.random.default_rng(6)
    T, k, n, H = 3, 2, 5, 8
    slot = np.array([[4, 1], [-1, 0], [2, 9]])
    y, w, do = g.standard_normal((n, H)), g.standard_normal((T, k)), g.standard_normal((T, H))
    dy, dw = rows.combine_rows_backward(do, y, w, slot)
    value = lambda yy, ww: (rows.combine_rows(yy, ww, slot) * do).sum()  # noqa: E731
    h = 1e-5
    for a, d, at in ((y, dy, 0), (w, dw, 1)):
        for i in np.ndindex(a.shape):
            up, dn = a.copy(), a.copy()
            up[i] += h
            dn[i] -= h
            p, m = ((up, w), (dn, w)) if at == 0 else ((y, up), (y, dn))
            assert abs((value(*p) - value(*m)) / (2 * h) - d[i]) < 1e-7
    assert (dy[3] == 0).all() and dw[1, 0] == 0 and dw[2, 1] == 0


def test_lora_by_hand():
    x = np.array([[1.0, 2.0], [3.0, 4.0], [5.0, 6.0]])
    a = np.array([[[1.0, 0.0]], [[0.0, 1.0]]])          # [2, 1, 2]
    b = np.array([[[1.0], [0.0], [2.0]], [[0.0], [1.0], [0.0]]])  # [2, 3, 1]
    out = rows.lora_add(np.ones((3, 3)), x, a, b, np.array([1, -1, 0]), np.array([2.0, 0.5]))
    assert np.allclose(out, [[1, 1 + 0.5 * 2, 1], [1, 1, 1], [1 + 2 * 5, 1, 1 + 2 * 10]])
