"""Many short packed sequences beside a long one through the delta rule in fp32: runs of 64
tokens are numbered by the tokens there are, not by the longest sequence for each of them.
Bars as in test_delta_gpu.py."""
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import model_ref as ref
from tests.gpu_util import host, rel
from tests.test_delta_gpu import BAR, STATE, inputs

pytestmark = pytest.mark.gpu


def offsets(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


def run(x, init, do, dfinal, cu):
    o, final, kept = ssd.delta_scan_fwd(*x.values(), init, cu_seqlens=cu, return_checkpoints=True)
    return (o, final) + ssd.delta_scan_bwd(do, *x.values(), kept, dfinal, cu_seqlens=cu)


def wanted(x, init, do, dfinal, cu, n):
    o, final, _ = ref.delta_fwd(*map(host, x.values()), host(init), cu, n ** -0.5)
    return (o, final) + ref.delta_bwd(host(do), *map(host, x.values()), host(init), host(dfinal), cu, n ** -0.5)


@pytest.mark.parametrize("lengths", [[3] * 30 + [700] + [0, 1, 64, 65] * 5, [1000] + [0] * 40, [0] * 40 + [129], [64] * 9 + [200, 63]])
@pytest.mark.parametrize("p,n,dtype", [(5, 7, "f32"), (70, 12, "bf16"), (40, 200, "f32")])
def test_short_ones_beside_a_long_one(lengths, p, n, dtype):
    cu = offsets(lengths)
    x, init, do, dfinal = inputs(len(cu) + p, cu[-1], len(lengths), 1, 2, p, n, dtype)
    for i, (g, w) in enumerate(zip(run(x, init, do, dfinal, cu), wanted(x, init, do, dfinal, cu, n))):
        assert rel(host(g), w) <= (BAR[dtype] if g.dtype == torch.bfloat16 else STATE[dtype]), i


def test_sequences_by_the_longest_one_s_runs_pass_a_grid():
    """32768 sequences of a token or none behind one of 65536, 64 heads: 2^31 runs if each
    sequence had as many as the longest."""
    heads, behind = 64, 32767
    lengths = [65536] + [i % 2 for i in range(behind)]
    cu = offsets(lengths)
    x, init, do, dfinal = inputs(1, cu[-1], len(lengths), 1, heads, 1, 1, "f32")
    got = run(x, init, do, dfinal, cu)
    # the last of the long one's tokens, from the state before them, and the first ones behind it
    first, few = 65536 - 200, offsets([200] + lengths[1:300])
    state = ssd.delta_scan_fwd(*(t[None, :first] for t in x.values()), init[:1])[1]
    cut = lambda t: t[first:first + few[-1]]   # noqa: E731
    want = wanted({name: cut(t) for name, t in x.items()}, torch.cat([state, init[1:300]]), cut(do), dfinal[:300], few, 1)
    for i, w in enumerate(want):
        g = cut(got[i]) if i not in (1, 7) else got[i][:300]
        if i == 7:      # (the long one's own goes back to its beginning)
            g, w = g[1:], w[1:]
        assert rel(host(g), w) <= STATE["f32"], i
    empty = [i for i in range(1, len(lengths)) if lengths[i] == 0]
    assert torch.equal(got[7][empty], dfinal[empty]) and torch.equal(got[1][empty], init[empty])
