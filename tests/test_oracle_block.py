"""The block operators' oracle: gradients against central differences, and the
8-bit format's defining properties."""
import numpy as np
import pytest

from oracle import block_oracle as O


def _differences(f, x, h=1e-5):
    """d(sum of f)/dx by central differences."""
    g = np.zeros_like(x)
    for i in np.ndindex(*x.shape):
        a, b = x.copy(), x.copy()
        a[i] += h
        b[i] -= h
        g[i] = (f(a) - f(b)) / (2 * h)
    return g


# central differences err by h^2/6 times the third derivative (at most about
# 1e2 for these inputs) plus rounding, 2^-53 / h times the sum's size (at most 1e2)
TOL = 1e-10 / 6 * 1e2 + 2.0 ** -53 / 1e-5 * 1e2 * 4


@pytest.mark.parametrize("rows,cols", [(1, 1), (3, 2), (4, 7), (2, 33)])
def test_layer_norm_gradient(rows, cols):
    rng = np.random.default_rng(rows * 100 + cols)
    x, gamma, beta = rng.normal(size=(rows, cols)) * 2, rng.normal(size=cols), rng.normal(size=cols)
    dy = rng.normal(size=(rows, cols))
    eps = 0.1
    _, mean, rstd = O.layer_norm(x, gamma, beta, eps)
    dx, dg, db = O.layer_norm_grad(dy, x, gamma, mean, rstd)
    assert np.allclose(dx, _differences(lambda v: (O.layer_norm(v, gamma, beta, eps)[0] * dy).sum(), x), rtol=0, atol=TOL)
    assert np.allclose(dg, _differences(lambda v: (O.layer_norm(x, v, beta, eps)[0] * dy).sum(), gamma), rtol=0, atol=TOL)
    assert np.allclose(db, _differences(lambda v: (O.layer_norm(x, gamma, v, eps)[0] * dy).sum(), beta), rtol=0, atol=TOL)


@pytest.mark.parametrize("kind", ["none", "relu", "gelu_tanh", "gelu_erf"])
def test_linear_gradients_of_a_two_layer_chain(kind):
    rng = np.random.default_rng(7)
    T, I, F, D = 3, 4, 5, 2
    x, w1, b1 = rng.normal(size=(T, I)), rng.normal(size=(I, F)), rng.normal(size=F)
    w2, b2, res, dy = rng.normal(size=(F, D)), rng.normal(size=D), rng.normal(size=(T, D)), rng.normal(size=(T, D))

    def loss(x, w1, b1, w2, b2):
        h, _ = O.linear(x, w1, b1, kind)
        return (O.linear(h, w2, b2, "none", res)[0] * dy).sum()

    h, z = O.linear(x, w1, b1, kind)
    dw2, db2 = O.linear_grad_weight(h, dy)
    dz = O.linear_grad_input(dy, w2, kind, z)
    dw1, db1 = O.linear_grad_weight(x, dz)
    dx = O.linear_grad_input(dz, w1)
    for got, f, at in ((dx, lambda v: loss(v, w1, b1, w2, b2), x), (dw1, lambda v: loss(x, v, b1, w2, b2), w1),
                       (db1, lambda v: loss(x, w1, v, w2, b2), b1), (dw2, lambda v: loss(x, w1, b1, v, b2), w2),
                       (db2, lambda v: loss(x, w1, b1, w2, v), b2)):
        assert np.allclose(got, _differences(f, at), rtol=0, atol=TOL)


def test_act8_properties():
    rng = np.random.default_rng(3)
    x = (rng.normal(size=(5, 70)) * np.exp2(rng.integers(-30, 30, size=(5, 1)))).astype(np.float32).astype(np.float64)
    x[1, 32:64] = 0.0
    q, b = O.act8_pack(x)
    v = O.act8_unpack(q, b, 70)
    assert q.shape == (5, 96) and b.shape == (5, 3) and not q[:, 70:].any()
    step = np.exp2(b.astype(np.float64) - 133).repeat(32, axis=1)[:, :70]
    top = np.abs(np.concatenate([x, np.zeros((5, 26))], 1)).reshape(5, 3, 32).max(2)
    E = b.astype(int) - 127
    assert np.all((np.exp2(E) <= top) | (top == 0)) and np.all(top < np.exp2(E + 1.0))
    # half a step, or one where 127.5 .. 128 steps are held at 127
    assert np.all(np.abs(v - x) <= np.where(np.abs(x) > 127 * step, step, step / 2))
    # every value is a bf16 number: 8 significant bits
    m, _ = np.frexp(v)
    assert np.array_equal(m * 256, np.rint(m * 256))
    # reading back what was read back changes nothing
    q2, b2 = O.act8_pack(v)
    assert np.array_equal(O.act8_unpack(q2, b2, 70), v)


def test_act8_special_groups():
    x = np.zeros((1, 96))
    x[0, 3] = np.inf
    x[0, 40] = 2.0 ** -140
    x[0, 64:] = [(-1) ** i * 1.999 for i in range(32)]
    q, b = O.act8_pack(x)
    v = O.act8_unpack(q, b, 96)
    assert list(b[0]) == [255, 7, 127]
    assert np.all(np.isnan(v[0, :32])) and np.all(v[0, 32:64] == 0)
    assert set(q[0, 64:]) == {127, -127}
