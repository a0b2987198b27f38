"""The gated recurrent block on the GPU: forward, gradients, tokens one by one
and the 8-bit form against the block composed of the 64-bit references.

Bars: every one of the block's ~6 stored intermediates is rounded to bf16 (2^-8
at most, 1.7e-3 on average) and the roundings add up along the chain at random;
the stream itself is f32 and mostly the input: 1e-2 for its change, 3e-2 for
gradients, which pass the chain twice.  In 8 bits the rows behind both norms and
their weights carry E4M3's 2^-4 at most (2.6e-2 on average, each): 0.1."""
import numpy as np
import pytest
import torch

from state_space_model_chunked_gb300.gated_block import GatedBlock
from tests import layer_ref as ref
from tests.gpu_util import host, rel

pytestmark = pytest.mark.gpu

D, DI, DF, EPS = 96, 136, 160, 1e-5


def _params(block):
    return {k: host(getattr(block, k)) for k in ("norm1", "w_in", "b_in", "w_out", "norm2", "w_up", "b_up", "w_down")}


def _reference(q, stream, init, dout=None, dfinal=None):
    b, length, d = stream.shape
    s0 = stream.reshape(-1, d)
    cu = [length * i for i in range(b + 1)]
    n1, _, r1 = ref.norm_fwd(s0, None, q["norm1"], EPS)
    p, _ = ref.linear_fwd(n1, q["w_in"], q["b_in"])
    x, g, z = p[:, :DI], p[:, DI:2 * DI], p[:, 2 * DI:]
    h, _, final, _ = ref.gated_fwd(x, g, z, init, cu)
    n2, s, r2 = ref.norm_fwd(h @ q["w_out"].T, s0, q["norm2"], EPS)
    u, pre = ref.linear_fwd(n2, q["w_up"], q["b_up"], None, "gelu")
    out = s + u @ q["w_down"].T
    if dout is None:
        return out.reshape(stream.shape), final
    do = dout.reshape(-1, d)
    grads = {}
    du, grads["w_down"], _ = ref.linear_bwd(do, u, q["w_down"])
    dn2, grads["w_up"], grads["b_up"] = ref.linear_bwd(du, n2, q["w_up"], pre, "gelu")
    ds, grads["norm2"] = ref.norm_bwd(dn2, s, q["norm2"], r2, do)
    dh, grads["w_out"], _ = ref.linear_bwd(ds, h, q["w_out"])
    dx, dg, dz, dinit = ref.gated_bwd(dh, x, g, z, init, dfinal, cu)
    dn1, grads["w_in"], grads["b_in"] = ref.linear_bwd(np.concatenate([dx, dg, dz], axis=1), n1, q["w_in"])
    dstream, grads["norm1"] = ref.norm_bwd(dn1, s0, q["norm1"], r1, ds)
    return out.reshape(stream.shape), final, dstream.reshape(stream.shape), dinit, grads


def _inputs(b, length):
    gen = torch.Generator(device="cuda").manual_seed(b * 100 + length)
    new = lambda *s: torch.empty(s, device="cuda").normal_(generator=gen)   # noqa: E731
    return new(b, length, D), new(b, DI), new(b, length, D), new(b, DI)


@pytest.mark.parametrize("b,length", [(1, 1), (2, 37), (3, 200)])
def test_block_forward_and_gradients(b, length):
    block = GatedBlock.random(D, DI, DF, seed=length)
    stream, init, dout, dfinal = _inputs(b, length)
    out, final, saved = block.forward(stream, init)
    dstream, dinit, grads = block.backward(saved, dout, dfinal)
    outr, finalr, dsr, dir_, gr = _reference(_params(block), host(stream), host(init), host(dout), host(dfinal))
    assert rel(host(out) - host(stream), outr - host(stream)) <= 1e-2
    assert rel(host(final), finalr) <= 1e-2
    assert rel(host(dstream) - host(dout), dsr - host(dout)) <= 3e-2 and rel(host(dinit), dir_) <= 3e-2
    for k, v in gr.items():
        assert rel(host(grads[k]), v) <= 3e-2, k


@pytest.mark.parametrize("in_8_bits,bar", [(False, 1e-2), (True, 0.1)])
def test_block_token_by_token_and_in_8_bits(in_8_bits, bar):
    block = GatedBlock.random(D, 144, DF, seed=7)
    b, length = 2, 20
    stream = _inputs(b, length)[0]
    q = _params(block)
    global DI
    keep, DI = DI, 144
    try:
        outr, finalr = _reference(q, host(stream), np.zeros((b, 144)))
    finally:
        DI = keep
    run = block.in_8_bits() if in_8_bits else block
    out, final, saved = run.forward(stream, keep=False)
    assert saved is None
    assert rel(host(out) - host(stream), outr - host(stream)) <= bar and rel(host(final), finalr) <= bar
    state = torch.zeros((b, 144), device="cuda")
    for t in range(length):
        y = run.step(stream[:, t].contiguous(), state)
        assert rel(host(y) - host(stream[:, t]), outr[:, t] - host(stream[:, t])) <= 2 * bar
    assert rel(host(state), finalr) <= bar


def test_8_bit_block_refuses_to_train():
    block = GatedBlock.random(D, 144, DF).in_8_bits()
    with pytest.raises(ValueError):
        block.backward(None, None)
