"""The 64-bit reference's gradients against central differences of its forward
passes (step 1e-5 in 64 bits: truncation and rounding each near 1e-10)."""
import numpy as np
import pytest

from tests import layer_ref as ref

STEP, TOL = 1e-5, 1e-7


def _differences(loss, at):
    grad = np.empty_like(at)
    flat, out = at.reshape(-1), grad.reshape(-1)
    for i in range(flat.size):
        keep = flat[i]
        flat[i] = keep + STEP
        up = loss()
        flat[i] = keep - STEP
        out[i] = (up - loss()) / (2 * STEP)
        flat[i] = keep
    return grad


def _close(a, b):
    np.testing.assert_allclose(a, b, rtol=TOL, atol=TOL)


def test_norm_gradients():
    rng = np.random.default_rng(0)
    x, r = rng.standard_normal((3, 5)), rng.standard_normal((3, 5))
    w, dy, ds = rng.standard_normal(5), rng.standard_normal((3, 5)), rng.standard_normal((3, 5))

    def loss():
        y, s, _ = ref.norm_fwd(x, r, w, 1e-3)
        return (y * dy).sum() + (s * ds).sum()
    _, s, rstd = ref.norm_fwd(x, r, w, 1e-3)
    got, dw = ref.norm_bwd(dy, s, w, rstd, ds)
    _close(got, _differences(loss, x))
    _close(got, _differences(loss, r))
    _close(dw, _differences(loss, w))


@pytest.mark.parametrize("act", ["none", "silu", "gelu", "relu"])
def test_product_gradients(act):
    rng = np.random.default_rng(1)
    x, w, b = rng.standard_normal((4, 3)), rng.standard_normal((5, 3)), rng.standard_normal(5)
    dy = rng.standard_normal((4, 5))

    def loss():
        return (ref.linear_fwd(x, w, b, None, act)[0] * dy).sum()
    _, p = ref.linear_fwd(x, w, b, None, act)
    dx, dw, db = ref.linear_bwd(dy, x, w, p, act)
    _close(dx, _differences(loss, x))
    _close(dw, _differences(loss, w))
    _close(db, _differences(loss, b))


@pytest.mark.parametrize("gate", [False, True])
def test_recurrence_gradients(gate):
    rng = np.random.default_rng(2)
    cu = [0, 3, 3, 4, 9]
    x, g, z = (rng.standard_normal((9, 2)) for _ in range(3))
    z = z if gate else None
    init, dfinal = rng.standard_normal((4, 2)), rng.standard_normal((4, 2))
    dy = rng.standard_normal((9, 2))

    def loss():
        y, _, final, _ = ref.gated_fwd(x, g, z, init, cu)
        return (y * dy).sum() + (final * dfinal).sum()
    dx, dg, dz, dinit = ref.gated_bwd(dy, x, g, z, init, dfinal, cu)
    _close(dx, _differences(loss, x))
    _close(dg, _differences(loss, g))
    _close(dinit, _differences(loss, init))
    if gate:
        _close(dz, _differences(loss, z))
