"""Long sequences of few heads through the gated delta rule: they are walked in parts side by
side, and the states between the parts are joined by what a part makes of a unit matrix.
Against tests/model_ref.py, with memories that reach over the parts (little decay, small beta).
Bars as in test_delta_gpu.py: the state is held in fp32, and what a chunk adds to it, or a
joining product, is off by at most 3e-5 of what it adds.
"""
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import model_ref as ref
from tests.gpu_util import host, rel
from tests.test_delta_gpu import BAR, STATE, inputs

pytestmark = pytest.mark.gpu


def sequences(lengths):
    cu = [0]
    for n in lengths:
        cu.append(cu[-1] + n)
    return cu


def remembered(*args):
    x, init, do, dfinal = inputs(*args, forget=0.001)
    x["beta"] *= 0.1
    return x, init, do, dfinal


PARTS = [  # lengths, groups, heads, headdim, dstate
    ([3100], 1, 1, 128, 128), ([5000], 1, 2, 64, 64), ([16 * 1024 + 5], 1, 1, 24, 72), ([3200], 1, 2, 136, 128),
    ([0, 4100, 64, 12300, 1], 1, 2, 72, 40), ([3136, 3136], 2, 2, 64, 104), ([4200], 16, 32, 8, 16)]


@pytest.mark.parametrize("lengths,groups,heads,p,n", PARTS)
@pytest.mark.parametrize("start", [False, True])
def test_forward_in_parts(lengths, groups, heads, p, n, start):
    cu = sequences(lengths)
    x, init, _, _ = remembered(sum(lengths) + p, cu[-1], len(lengths), groups, heads, p, n, "bf16")
    run = lambda: ssd.delta_scan_fwd(*x.values(), init if start else None, cu_seqlens=cu,     # noqa: E731
                                     return_checkpoints=True)
    o, final, kept = run()
    want, last, before = ref.delta_fwd(*map(host, x.values()), host(init) * start, cu, n ** -0.5)
    assert rel(host(o), want) <= BAR["bf16"]
    assert rel(host(final), last) <= STATE["bf16"]
    for place, state in ref.delta_kept(before, cu):
        assert rel(host(kept[place]), state) <= STATE["bf16"]
    again = run()
    assert all(torch.equal(a, b) for a, b in zip((o, final), again[:2]))


def test_growth_and_resets_in_parts():
    """Parts that reset the state altogether, and parts in which it grows."""
    x, init, _, _ = remembered(5, 4096, 1, 1, 2, 128, 128, "bf16")
    x["g"][1500, 0] = float("-inf")
    x["g"][2900:3000] = 0.01
    o, final = ssd.delta_scan_fwd(*(t[None] for t in x.values()), init)
    want, last, _ = ref.delta_fwd(*map(host, x.values()), host(init), [0, 4096], 128 ** -0.5)
    assert rel(host(o[0]), want) <= BAR["bf16"]
    assert rel(host(final), last) <= STATE["bf16"]


BACK = [([1700], 1, 1, 128, 128), ([1540], 2, 4, 64, 64), ([3000], 1, 1, 24, 72), ([0, 1600, 64, 4500, 1], 1, 2, 40, 40),
        ([3100], 16, 32, 8, 16), ([3200], 1, 2, 64, 64), ([700, 2500, 900], 2, 2, 128, 64)]


@pytest.mark.parametrize("lengths,groups,heads,p,n", BACK)
@pytest.mark.parametrize("behind", [False, True])
def test_gradients_in_parts(lengths, groups, heads, p, n, behind):
    cu = sequences(lengths)
    x, init, do, dfinal = remembered(sum(lengths) + n, cu[-1], len(lengths), groups, heads, p, n, "bf16")
    _, _, kept = ssd.delta_scan_fwd(*x.values(), init, cu_seqlens=cu, return_checkpoints=True)
    run = lambda: ssd.delta_scan_bwd(do, *x.values(), kept, dfinal if behind else None, cu_seqlens=cu)   # noqa: E731
    got = run()
    want = ref.delta_bwd(host(do), *map(host, x.values()), host(init), host(dfinal) * behind, cu, n ** -0.5)
    for name, a, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dinit"), got, want):
        assert rel(host(a).reshape(w.shape), w) <= (BAR["bf16"] if a.dtype == torch.bfloat16 else STATE["bf16"]), name
    assert all(torch.equal(a, b) for a, b in zip(got, run()))


def test_the_final_state_in_the_initial_one_s_place():
    for length, heads in ((3200, 1), (200, 2)):
        x, init, _, _ = remembered(7, length, 1, 1, heads, 128, 64, "bf16")
        b = [t[None] for t in x.values()]
        o, final = ssd.delta_scan_fwd(*b, init)
        state = init.clone()
        o2, same = ssd.delta_scan_fwd(*b, state, final_state=state)
        assert same is state and torch.equal(o, o2) and torch.equal(final, state)


def test_two_graphs_with_one_workspace():
    """Captured on another stream and replayed in turns, with new inputs in the old places."""
    x, init, _, _ = remembered(8, 3300, 1, 1, 2, 64, 128, "bf16")
    y, init2, _, _ = remembered(9, 3300, 1, 1, 2, 64, 128, "bf16")
    both = [([t[None].clone() for t in x.values()], init.clone()), ([t[None].clone() for t in y.values()], init2.clone())]
    want = [ssd.delta_scan_fwd(*b, i) for b, i in both]
    need = ssd.delta_scan_workspace_bytes(torch.bfloat16, 3300, 1, 2, 64, 128, 1)
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    graphs, got = [], []
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for b, i in both:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got.append(ssd.delta_scan_fwd(*b, i, workspace=ws))
        graphs.append(graph)
    torch.cuda.current_stream().wait_stream(side)
    for turn in (0, 1, 0, 1):
        for t in got[turn]:
            t.fill_(7.0)
        graphs[turn].replay()
        assert all(torch.equal(a, w) for a, w in zip(got[turn], want[turn]))
    for old, new in zip(both[0][0] + [both[0][1]], both[1][0] + [both[1][1]]):
        old.copy_(new)
    graphs[0].replay()
    assert all(torch.equal(a, w) for a, w in zip(got[0], want[1]))


def test_offsets_beyond_32_bits():
    """Values past the 2^31st: a sequence behind a long one, against the same by itself."""
    tokens, tail, heads = 270000, 700, 64
    unit = lambda *s: torch.nn.functional.normalize(torch.randn(*s, device="cuda"), dim=-1).bfloat16()  # noqa: E731
    x = [unit(tokens, 2, 64), unit(tokens, 2, 64), torch.randn((tokens, heads, 128), device="cuda", dtype=torch.bfloat16),
         -0.1 * torch.rand((tokens, heads), device="cuda"), torch.rand((tokens, heads), device="cuda")]
    assert x[2].numel() > 2 ** 31
    o, final = ssd.delta_scan_fwd(*x, cu_seqlens=[0, tokens - tail, tokens])
    o2, final2 = ssd.delta_scan_fwd(*(t[None, tokens - tail:].clone() for t in x))
    assert torch.equal(o[tokens - tail:], o2[0]) and torch.equal(final[1], final2[0])
