"""The recurrence where its gates nearly close: f and 1 - f each keep a precision of
their own, also where the one that is near zero is all that a result is made of.

Bars, derived before the first run.  f comes from the hardware's exponential of a
rounded argument: |g| 2^-24 + 4 * 2^-23 of itself, and a token's multiplications add
2 * 2^-23.  A result that is a product of j such factors errs by at most
j (|g| 2^-24 + 6 * 2^-23), below 1e-5 for j <= 5 and |g| <= 20; every token is held to
1e-5 of its own size."""
import numpy as np
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import layer_ref as ref
from tests.gpu_util import host

pytestmark = pytest.mark.gpu
BAR = 1e-5


def _values(rng, *shape):
    return torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).cuda()


def _each_row(got, want, rows):
    for t in rows:
        wrong = np.linalg.norm(got[t] - want[t])
        assert wrong <= BAR * np.linalg.norm(want[t]), (t, wrong / np.linalg.norm(want[t]))


@pytest.mark.parametrize("length", [3, 5, 10, 66, 130, 450])
@pytest.mark.parametrize("gate", [-9.0, -12.0, -18.0])
@pytest.mark.parametrize("width", [64, 33])
def test_gradient_of_the_last_token_alone(length, gate, width):
    """Earlier tokens' gradients are products of closed gates (f), across warps' and tiles' ends too."""
    rng = np.random.default_rng(length)
    x, init = _values(rng, length, width), _values(rng, 1, width)
    g = gate + 0.2 * _values(rng, length, width)
    dy = torch.zeros_like(x)
    dy[-1] = _values(rng, width)
    _, _, kept = ssd.gated_scan_fwd(x[None], g[None], None, init, return_checkpoints=True)
    dx, dg, _, dinit = ssd.gated_scan_bwd(dy[None], x[None], g[None], kept, None, init)
    dxr, dgr, _, dir_ = ref.gated_bwd(host(dy), host(x), host(g), None, host(init), np.zeros((1, width)), [0, length])
    last = range(length - 1, max(length - 5, -1), -1)
    _each_row(host(dx)[0], dxr, last)
    # x and the state before it are of one size here, so their difference is exact to a few 2^-23 of it
    _each_row(host(dg)[0], dgr, last)
    if length <= 4:
        _each_row(host(dinit), dir_, [0])
    ssd.last_device_error()


@pytest.mark.parametrize("start", [0, 1, 5, 60, 63])
@pytest.mark.parametrize("gate", [-9.0, -12.0, -18.0])
@pytest.mark.parametrize("width", [64, 33])
def test_state_that_outweighs_the_inputs(start, gate, width):
    """Inputs of zero behind a state: what is left of it is a product of closed gates, in y, dz and dg alike."""
    rng = np.random.default_rng(start)
    length, after = start + 5, slice(start, start + 4)
    x, z, dy = (_values(rng, length, width) for _ in range(3))
    g = _values(rng, length, width)
    x[after], g[after] = 0.0, gate + 0.2 * g[after]
    init = _values(rng, 1, width)
    y, _, kept = ssd.gated_scan_fwd(x[None], g[None], z[None], init, return_checkpoints=True)
    _, dg, dz, _ = ssd.gated_scan_bwd(dy[None], x[None], g[None], kept, z[None], init)
    hx, hg, hz, hi = host(x), host(g), host(z), host(init)
    yr = ref.gated_fwd(hx, hg, hz, hi, [0, length])[0]
    _, dgr, dzr, _ = ref.gated_bwd(host(dy), hx, hg, hz, hi, np.zeros((1, width)), [0, length])
    rows = range(start, start + 4)
    _each_row(host(y)[0], yr, rows)
    _each_row(host(dz)[0], dzr, rows)
    _each_row(host(dg)[0], dgr, rows)
    ssd.last_device_error()


def _bound(v, more=0):
    """What sigmoid(v) may err by, of itself: |v| log2 e is one rounded product with a
    rounded constant (1.22 |v| 2^-24 of the exponential), the hardware's exponential errs by
    2^-22, its reciprocal by 2^-23, and two roundings come after; `more` of 2^-24."""
    return (1.25 * np.abs(v) + 8 + more) * 2.0 ** -24


def test_gates_value_by_value():
    g = torch.cat([torch.linspace(-80, 80, 40001), torch.linspace(-1, 1, 4001)]).cuda()[None]
    one, zero = torch.ones_like(g), torch.zeros_like(g)
    keep, drop = one.clone(), zero.clone()
    ssd.gated_state_update(keep, zero, g)              # f * 1 + (1 - f) * 0
    ssd.gated_state_update(drop, one, g)               # f * 0 + (1 - f) * 1
    v = host(g)
    assert np.all(np.abs(host(keep) - ref.sigmoid(v)) <= _bound(v) * ref.sigmoid(v))
    assert np.all(np.abs(host(drop) - ref.sigmoid(-v)) <= _bound(v) * ref.sigmoid(-v))


def test_silu_value_by_value():
    p = torch.linspace(-80, 80, 40001).cuda()[:, None]
    y = ssd.linear_fwd(p, torch.ones((1, 1), device="cuda"), activation="silu")
    v = host(p)
    assert np.all(np.abs(host(y) - ref.silu(v)) <= _bound(v, 1) * np.abs(ref.silu(v)))
    z, h = p.T.contiguous(), torch.ones((1, 40001), device="cuda")
    big = torch.full_like(z, 80.0)                     # f = 1: the state stays 1
    y = ssd.gated_state_update(h, torch.zeros_like(z), big, z)
    assert np.all(np.abs(host(y) - ref.silu(v.T)) <= _bound(v.T, 1) * np.abs(ref.silu(v.T)))
