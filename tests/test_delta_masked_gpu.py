"""Tokens that the delta rule's beta masks: what their values hold, of any size, reaches no
other token and no gradient but their own beta's.  Bars as in test_delta_gpu.py."""
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import model_ref as ref
from tests.gpu_util import host, rel
from tests.test_delta_gpu import BAR, STATE, inputs

pytestmark = pytest.mark.gpu

NAMES = ("dq", "dk", "dv", "dg", "dbeta", "dinit")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("size", [1e8, 1e30])
@pytest.mark.parametrize("cu,groups,heads,p,n", [([0, 140], 1, 2, 64, 128), ([0, 70, 70, 200], 2, 4, 128, 64), ([0, 1700], 1, 1, 64, 64)])
def test_values_that_beta_masks(cu, groups, heads, p, n, size, dtype):
    x, init, do, dfinal = inputs(p + n, cu[-1], len(cu) - 1, groups, heads, p, n, dtype)
    masked = torch.zeros(cu[-1], dtype=torch.bool)
    masked[20:40] = masked[90] = masked[-1] = True
    x["beta"][masked] = 0.0
    x["v"][masked] *= size
    o, final, kept = ssd.delta_scan_fwd(*x.values(), init, cu_seqlens=cu, return_checkpoints=True)
    want, last, _ = ref.delta_fwd(*map(host, x.values()), host(init), cu, n ** -0.5)
    assert rel(host(o), want) <= BAR[dtype] and rel(host(final), last) <= STATE[dtype]
    got = ssd.delta_scan_bwd(do, *x.values(), kept, dfinal, cu_seqlens=cu)
    grad = ref.delta_bwd(host(do), *map(host, x.values()), host(init), host(dfinal), cu, n ** -0.5)
    for name, g, w in zip(NAMES, map(host, got), grad):
        bar = BAR[dtype] if name in ("dq", "dk", "dv") else STATE[dtype]
        if name == "dinit":
            assert rel(g, w) <= bar, name
            continue
        assert rel(g[~masked.numpy()], w[~masked.numpy()]) <= bar, name
        if w[masked.numpy()].any():         # (of v they are zeros; of beta as large as the values)
            assert rel(g[masked.numpy()], w[masked.numpy()]) <= bar, name


def test_a_large_value_by_a_tiny_beta():
    """Their product is what counts: 1e-20 of 1e19."""
    x, init, do, dfinal = inputs(3, 100, 1, 1, 2, 64, 64, "bf16")
    x["beta"][30, 0], x["beta"][70, 1] = 1e-20, -1e-20
    x["v"][30, 0] *= 1e19
    x["v"][70, 1] *= 1e19
    b = [t[None] for t in x.values()]
    o, final, kept = ssd.delta_scan_fwd(*b, init, return_checkpoints=True)
    want, last, _ = ref.delta_fwd(*map(host, x.values()), host(init), [0, 100], 0.125)
    assert rel(host(o)[0], want) <= BAR["bf16"] and rel(host(final), last) <= STATE["bf16"]
    got = ssd.delta_scan_bwd(do[None], *b, kept, dfinal)
    grad = ref.delta_bwd(host(do), *map(host, x.values()), host(init), host(dfinal), [0, 100], 0.125)
    for name, g, w in zip(NAMES, got, grad):
        g = host(g).reshape(w.shape)
        if name == "dbeta":
            for t, h in ((30, 0), (70, 1)):
                assert abs(g[t, h] - w[t, h]) <= STATE["bf16"] * abs(w[t, h])
                g[t, h] = w[t, h] = 0.0
        assert rel(g, w) <= (BAR["bf16"] if name in ("dq", "dk", "dv") else STATE["bf16"]), name
