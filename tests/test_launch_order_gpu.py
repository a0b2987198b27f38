"""A kernel's launch and set-up may run while the one in front of it in the stream
ends; nothing it reads or writes may.  Chains in which every call reads what the one
before wrote, in place where it can be, give bit for bit what they give with the
device idle between calls."""
import numpy as np
import pytest
import torch

import state_space_model_chunked_gb300 as ssd

pytestmark = pytest.mark.gpu


def _tens(rng, *shape, dtype=torch.bfloat16, std=1.0):
    return torch.from_numpy((rng.standard_normal(shape) * std).astype(np.float32)).cuda().to(dtype)


def _same(run):
    """run(pause): the outputs of a chain, pause() between its calls."""
    apart = run(torch.cuda.synchronize)
    torch.cuda.synchronize()
    for _ in range(5):
        together = run(lambda: None)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(apart, together))


@pytest.mark.parametrize("tokens", [1, 4, 16, 40, 200])
@pytest.mark.parametrize("width", [264, 2560])
def test_decode_chain(tokens, width):
    rng = np.random.default_rng(tokens + width)
    wn = _tens(rng, width, dtype=torch.float32)
    wi, wo = _tens(rng, 3 * width, width, std=width ** -0.5), _tens(rng, width, width, std=width ** -0.5)
    start = _tens(rng, tokens, width, dtype=torch.float32)

    def run(pause):
        stream, state, seen = start.clone(), torch.zeros(tokens, width, device="cuda"), []
        for _ in range(12):
            n, stream, _, _ = ssd.rmsnorm_fwd(stream.bfloat16(), wn, stream, residual_out=stream)
            pause()
            p = ssd.linear_fwd(n, wi)
            pause()
            y = ssd.gated_state_update(state, p[:, :width], p[:, width:2 * width], p[:, 2 * width:])
            pause()
            r = ssd.linear_fwd(y, wo, residual=n)
            pause()
            n, stream, _, _ = ssd.rmsnorm_fwd(r, wn, stream, residual_out=stream)
            pause()
            seen += [n, r]
        return seen + [stream, state]
    _same(run)


@pytest.mark.parametrize("rows,width,features", [(40, 264, 520), (900, 1024, 2048), (2500, 2560, 512)])
def test_training_chain(rows, width, features):
    rng = np.random.default_rng(rows)
    wn, w = _tens(rng, width, dtype=torch.float32), _tens(rng, features, width, std=width ** -0.5)
    back = _tens(rng, features, features, std=features ** -0.5)
    x, r0 = _tens(rng, rows, width), _tens(rng, rows, width, dtype=torch.float32)

    def run(pause):
        out, dy = [], None
        for _ in range(4):
            n, s, rstd, _ = ssd.rmsnorm_fwd(x, wn, r0)
            pause()
            y, pre = ssd.linear_fwd(n, w, activation="silu", return_preact=True)
            pause()
            dy = ssd.linear_fwd(y, back)
            pause()
            dn, dw, db = ssd.linear_bwd(dy, n, w, pre, activation="silu")
            pause()
            dx, ds, dwn = ssd.rmsnorm_bwd(dn, s, wn, rstd)[:3]
            pause()
            e, dw2, db2 = ssd.linear_bwd(dy, n, w)
            pause()
            out += [dw, db, dx, dwn, e, dw2, db2]
        return [t for t in out if t is not None]
    _same(run)
