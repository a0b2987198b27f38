"""How far a token's NaN or infinity reaches in the delta rule: what the formula says, and where
runs of 64 tokens are taken together (the tensor cores' outputs, all gradients) its own run."""
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests.test_delta_gpu import batched, inputs

pytestmark = pytest.mark.gpu

T, RUN, NEXT = 100, 64, 128         # the token, its run's first one, and the next run's


def same(a, b):
    return torch.equal(a, b) and torch.isfinite(a.float()).all()


@pytest.mark.parametrize("value", [float("nan"), float("inf")])
@pytest.mark.parametrize("which", ["v", "k", "q", "g", "beta"])
@pytest.mark.parametrize("dtype,p,n", [("bf16", 64, 128), ("bf16", 128, 64), ("f32", 64, 64)])
def test_outputs(dtype, p, n, which, value):
    x, init, _, _ = inputs(6, 200, 1, 2, 4, p, n, dtype)
    clean = ssd.delta_scan_fwd(*batched(x, 1).values(), init, return_checkpoints=True)
    if which == "v":
        x["v"][T, 1, 3] = value
    elif which in "kq":
        x[which][T, 0, 5] = value           # of heads 0 and 1
    else:
        x[which][T, 1] = value
    o, final, kept = ssd.delta_scan_fwd(*batched(x, 1).values(), init, return_checkpoints=True)
    before = T if dtype == "f32" else RUN
    assert same(o[0, :before], clean[0][0, :before])
    others = [2, 3] + ([0] if which not in "kq" else [])        # heads
    assert same(o[:, :, others], clean[0][:, :, others]) and same(final[:, others], clean[1][:, others])
    assert same(kept[:2], clean[2][:2])                         # the states before tokens 0 and 64
    if which == "v":                                            # the state's other rows
        rows = [i for i in range(p) if i != 3]
        assert same(o[:, :, 1, rows], clean[0][:, :, 1, rows])
        assert not torch.isfinite(o[0, T:, 1, 3].float()).any()
    if which == "q":
        assert same(final, clean[1]) and same(o[0, NEXT:], clean[0][0, NEXT:])
    assert not torch.isfinite(o[0, T, 1].float()).all()


@pytest.mark.parametrize("dtype,p,n", [("bf16", 64, 128), ("bf16", 128, 64), ("f32", 64, 64)])
def test_gradients(dtype, p, n):
    x, init, do, dfinal = inputs(7, 200, 1, 2, 4, p, n, dtype)
    b = batched(x, 1)
    kept = ssd.delta_scan_fwd(*b.values(), init, return_checkpoints=True)[2]
    clean = ssd.delta_scan_bwd(do[None], *b.values(), kept, dfinal)
    do[T, 1, 3] = float("nan")
    got = ssd.delta_scan_bwd(do[None], *b.values(), kept, dfinal)
    for i, (g, w) in enumerate(zip(got, clean)):
        heads = [2, 3] if i > 1 else [1]            # dq and dk by groups: of two heads each
        at = (slice(None), heads) if i == 5 else (slice(None), slice(None), heads)
        assert same(g[at], w[at])
        if i < 5:
            assert same(g[:, NEXT:], w[:, NEXT:])
