"""The product's two gradients where one launch computes both: tiles of more than one
round of the machine, the longer sum over tokens or over features, and last tiles
that are not full, against the formulas in 64 bits.  A bf16 result is rounded once,
by at most 2^-8 of itself; the bar adds 1e-4 for the sums' 32 bits."""
import numpy as np
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import layer_ref as ref

pytestmark = pytest.mark.gpu
BAR = 2.0 ** -8 + 1e-4


def _values(rng, rows, cols, pad=0):
    t = torch.from_numpy(rng.standard_normal((rows, cols + pad), dtype=np.float32))
    return t.cuda().bfloat16()[:, :cols]


def _wrong(got, want):
    return float(np.linalg.norm(got.double().cpu().numpy() - want) / np.linalg.norm(want))


@pytest.mark.parametrize("tokens,features,inner", [
    (100, 264, 72),         # one tile of each, neither full
    (300, 1024, 1000),
    (2635, 7664, 1952),     # the sum over features is the longer, 88 and 240 tiles
    (9000, 520, 264),       # the sum over tokens is the longer, 6 and 72 tiles
    (5000, 2056, 1032),
    (2500, 5000, 2600),
])
@pytest.mark.parametrize("pad", [0, 24])
def test_gradients_together(tokens, features, inner, pad):
    rng = np.random.default_rng(tokens + features + inner + pad)
    x, dy = _values(rng, tokens, inner, pad), _values(rng, tokens, features, pad)
    w = _values(rng, features, inner)
    dx, dw, db = ssd.linear_bwd(dy, x, w)
    host = [t.double().cpu().numpy() for t in (dy, x, w)]
    dxr, dwr, dbr = ref.linear_bwd(*host)
    assert _wrong(dx, dxr) <= BAR and _wrong(dw, dwr) <= BAR
    # no tile is left out or computed for another: the largest error of one value
    for got, want in ((dx, dxr), (dw, dwr)):
        worst = np.abs(got.double().cpu().numpy() - want).max()
        assert worst <= BAR * np.abs(want).max()
    assert np.linalg.norm(db.double().cpu().numpy() - dbr) <= 1e-5 * np.linalg.norm(host[0])
    again = ssd.linear_bwd(dy, x, w)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1]) and torch.equal(db, again[2])


def test_gradients_with_an_infinite_value_elsewhere():
    """A row of dy that is not finite reaches its row of dx and every row of dw that
    its column stands for, and nothing else."""
    rng = np.random.default_rng(3)
    x, dy, w = _values(rng, 700, 520), _values(rng, 700, 1288), _values(rng, 1288, 520)
    dy[650, 1280] = float("inf")
    dx, dw, _ = ssd.linear_bwd(dy, x, w)
    rows = (~torch.isfinite(dx.float()).all(dim=1)).nonzero().flatten().tolist()
    cols = (~torch.isfinite(dw.float()).all(dim=1)).nonzero().flatten().tolist()
    assert rows == [650] and cols == [1280]


@pytest.mark.parametrize("act", ["none", "silu"])
def test_calls_in_a_row_share_a_workspace(act):
    """The bias's sum runs beside the products; the next call's writes to the same
    workspace wait for it."""
    rng = np.random.default_rng(8)
    x, w = _values(rng, 1500, 264), _values(rng, 2048, 264)
    calls = [(_values(rng, 1500, 2048), _values(rng, 1500, 2048) if act != "none" else None) for _ in range(8)]
    alone = []
    for dy, p in calls:
        alone.append(ssd.linear_bwd(dy, x, w, p, activation=act))
        torch.cuda.synchronize()
    need = ssd.linear_bwd_workspace_bytes(torch.bfloat16, 1500, 2048, 264, act)
    work = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    together = [ssd.linear_bwd(dy, x, w, p, activation=act, workspace=work) for dy, p in calls]
    for one, other in zip(alone, together):
        assert all(torch.equal(a, b) for a, b in zip(one, other))
