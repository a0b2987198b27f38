"""The plain implementations of tests/model_ref.py: gradients against central
differences of the forward passes, and what the formulas imply."""
import numpy as np
import pytest

from tests import model_ref as ref

H = 1e-5


def difference(f, x, at):
    up, down = x.copy(), x.copy()
    up[at] += H
    down[at] -= H
    return (f(up) - f(down)) / (2 * H)


def check(f, x, grad, rng, count=12):
    for _ in range(count):
        at = tuple(int(rng.integers(n)) for n in x.shape)
        d = difference(f, x, at)
        assert abs(d - grad[at]) <= 1e-6 * max(1.0, abs(d))


def test_layernorm_gradients():
    rng = np.random.default_rng(0)
    x, w, b, dy = rng.standard_normal((3, 7)) + 2, rng.standard_normal(7), rng.standard_normal(7), rng.standard_normal((3, 7))
    y, s, mean, rstd = ref.layernorm_fwd(x, None, w, b, 1e-3)
    ds, dw, db = ref.layernorm_bwd(dy, s, w, mean, rstd, None)
    check(lambda t: (ref.layernorm_fwd(t, None, w, b, 1e-3)[0] * dy).sum(), x, ds, rng)
    check(lambda t: (ref.layernorm_fwd(x, None, t, b, 1e-3)[0] * dy).sum(), w, dw, rng)
    check(lambda t: (ref.layernorm_fwd(x, None, w, t, 1e-3)[0] * dy).sum(), b, db, rng)


def test_embedding_gradient():
    rng = np.random.default_rng(1)
    table, tokens = rng.standard_normal((5, 3)), np.array([[4, 0, -1, 4], [2, 5, 4, 0]])
    dy = rng.standard_normal((2, 4, 3))
    assert np.all(ref.embedding_fwd(tokens, table, 2.0)[0, 2] == 0) and np.all(ref.embedding_fwd(tokens, table, 2.0)[1, 1] == 0)
    check(lambda t: (ref.embedding_fwd(tokens, t, 2.0) * dy).sum(), table, ref.embedding_bwd(dy, tokens, 5, 2.0), rng)


@pytest.mark.parametrize("cu", [[0, 6], [0, 2, 2, 7]])
def test_delta_gradients(cu):
    rng = np.random.default_rng(len(cu))
    T, G, heads, P, N, n = cu[-1], 2, 4, 3, 5, len(cu) - 1
    x = dict(q=rng.standard_normal((T, G, N)), k=rng.standard_normal((T, G, N)) * 0.4, v=rng.standard_normal((T, heads, P)),
             g=-rng.random((T, heads)), beta=rng.random((T, heads)), init=rng.standard_normal((n, heads, P, N)))
    do, dfinal = rng.standard_normal((T, heads, P)), rng.standard_normal((n, heads, P, N))
    grads = ref.delta_bwd(do, *x.values(), dfinal, cu, 0.7)
    for name, grad in zip(x, grads):
        def loss(t, name=name):
            o, final, _ = ref.delta_fwd(*dict(x, **{name: t}).values(), cu, 0.7)
            return (o * do).sum() + (final * dfinal).sum()
        check(loss, x[name], grad, rng)


def test_delta_rule_writes_what_a_key_then_reads():
    """With beta 1, no decay and a key of unit length, the state answers the key with the value."""
    rng = np.random.default_rng(3)
    k = rng.standard_normal((4, 1, 6))
    k /= np.linalg.norm(k, axis=-1, keepdims=True)
    v = rng.standard_normal((4, 1, 5))
    o, _, _ = ref.delta_fwd(k, k, v, np.zeros((4, 1)), np.ones((4, 1)), rng.standard_normal((1, 1, 5, 6)), [0, 4], 1.0)
    np.testing.assert_allclose(o, v, atol=1e-12)
