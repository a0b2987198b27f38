"""The gated delta rule on the GPU against tests/model_ref.py, on the inputs as the GPU
holds them.  Bars as relative L2, derived before the first run:
  bf16 outputs   rounded once, by at most 2^-8 of a value (3.91e-3), with below 1e-4 in
                 front: 4e-3.
  f32 outputs of f32 inputs   fp32 sums of up to 256 products along a memory of some 10^2
                 tokens: 1e-5.
  f32 outputs of bf16 inputs  where the tensor cores take them, factors that are no bf16
                 values are held in two parts, off by at most 2^-18 of themselves, the
                 products of both second parts (2^-16 of a term, at most) left out; of the
                 three such products that follow each other none adds more than
                 2^-18 + 2^-18 + 2^-16 in the worst case, of which sums of independent
                 terms keep a third: 3e-5.
"""
import numpy as np
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import model_ref as ref
from tests.gpu_util import host, rel

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BAR = {"f32": 1e-5, "bf16": 4e-3}
STATE = {"f32": 1e-5, "bf16": 3e-5}


def dev(a, dtype="f32"):
    return torch.from_numpy(np.asarray(a, dtype=np.float32)).to(DT[dtype]).cuda()


def inputs(seed, tokens, nseq, groups, heads, p, n, dtype, forget=1.0):
    rng = np.random.default_rng(seed)
    unit = lambda t: t / np.maximum(np.linalg.norm(t, axis=-1, keepdims=True), 1e-6)   # noqa: E731
    x = dict(q=dev(unit(rng.standard_normal((tokens, groups, n))), dtype),
             k=dev(unit(rng.standard_normal((tokens, groups, n)) + 0.3), dtype),
             v=dev(rng.standard_normal((tokens, heads, p)), dtype),
             g=dev(-forget * rng.random((tokens, heads)) ** 4), beta=dev(rng.random((tokens, heads))))
    init = dev(0.3 * rng.standard_normal((nseq, heads, p, n)))
    do = dev(rng.standard_normal((tokens, heads, p)), dtype)
    return x, init, do, dev(rng.standard_normal((nseq, heads, p, n)))


def batched(x, nseq):
    return {name: t.unflatten(0, (nseq, -1)) for name, t in x.items()}


SHAPES = [  # tokens a sequence, sequences, groups, heads, headdim, dstate
    (1, 1, 1, 1, 1, 1), (3, 2, 1, 2, 5, 7), (64, 1, 2, 4, 16, 32), (65, 2, 1, 1, 64, 64), (130, 1, 2, 2, 128, 128),
    (127, 3, 2, 4, 128, 64), (200, 2, 1, 3, 64, 128), (300, 1, 1, 1, 40, 200), (63, 1, 1, 2, 130, 20), (257, 1, 1, 2, 33, 256),
    (192, 2, 1, 2, 96, 112), (577, 1, 1, 1, 128, 128),
    (100, 1, 1, 2, 136, 8), (129, 1, 2, 2, 256, 72), (2, 3, 1, 1, 8, 128)]


@pytest.mark.parametrize("length,nseq,groups,heads,p,n", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_forward(length, nseq, groups, heads, p, n, dtype):
    x, init, _, _ = inputs(length + p, length * nseq, nseq, groups, heads, p, n, dtype)
    cu = [length * i for i in range(nseq + 1)]
    o, final, kept = ssd.delta_scan_fwd(*batched(x, nseq).values(), init, return_checkpoints=True)
    assert o.shape == (nseq, length, heads, p) and o.dtype == DT[dtype]
    want, last, before = ref.delta_fwd(*map(host, x.values()), host(init), cu, n ** -0.5)
    assert rel(host(o).reshape(want.shape), want) <= BAR[dtype]
    assert rel(host(final), last) <= STATE[dtype]
    assert kept.shape[0] == ssd.delta_scan_checkpoints(length * nseq, nseq)
    for place, state in ref.delta_kept(before, cu):
        assert rel(host(kept[place]), state) <= STATE[dtype]


@pytest.mark.parametrize("length,nseq,groups,heads,p,n", SHAPES)
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward(length, nseq, groups, heads, p, n, dtype):
    x, init, do, dfinal = inputs(length + p, length * nseq, nseq, groups, heads, p, n, dtype)
    cu = [length * i for i in range(nseq + 1)]
    b = batched(x, nseq)
    _, _, kept = ssd.delta_scan_fwd(*b.values(), init, scale=0.3, return_checkpoints=True)
    got = ssd.delta_scan_bwd(do.unflatten(0, (nseq, -1)), *b.values(), kept, dfinal, scale=0.3)
    want = ref.delta_bwd(host(do), *map(host, x.values()), host(init), host(dfinal), cu, 0.3)
    for name, g, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dinit"), got, want):
        bar = BAR[dtype] if name in ("dq", "dk", "dv") else STATE[dtype]
        assert rel(host(g).reshape(w.shape), w) <= bar, name


@pytest.mark.parametrize("p,n", [(64, 128), (128, 128), (24, 40)])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_packed_sequences(p, n, dtype):
    """Sequences of many lengths, empty ones among them, as column ranges of one matrix."""
    cu = [0, 0, 1, 64, 64, 129, 330, 331, 395, 395]
    nseq, groups, heads = len(cu) - 1, 2, 4
    x, init, do, dfinal = inputs(p, cu[-1], nseq, groups, heads, p, n, dtype)
    wide = torch.zeros((cu[-1], 2 * groups * n + heads * p + 8), dtype=DT[dtype], device="cuda")
    grads = torch.full_like(wide, 7.0)
    cut = lambda m: (m[:, 8:8 + groups * n].unflatten(-1, (groups, n)),   # noqa: E731
                     m[:, 8 + groups * n:8 + 2 * groups * n].unflatten(-1, (groups, n)),
                     m[:, 8 + 2 * groups * n:].unflatten(-1, (heads, p)))
    for name, part in zip("qkv", cut(wide)):
        part.copy_(x[name])
        x[name] = part
    o, final, kept = ssd.delta_scan_fwd(*x.values(), init, cu_seqlens=cu, return_checkpoints=True)
    want, last, before = ref.delta_fwd(*map(host, x.values()), host(init), cu, n ** -0.5)
    assert rel(host(o), want) <= BAR[dtype] and rel(host(final), last) <= STATE[dtype]
    assert torch.equal(final[0], init[0]) and torch.equal(final[3], init[3])
    for place, state in ref.delta_kept(before, cu):
        assert rel(host(kept[place]), state) <= STATE[dtype]
    dq, dk, dv = cut(grads)
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda")
    got = ssd.delta_scan_bwd(do, *x.values(), kept, dfinal, cu_seqlens=cu, cu_seqlens_dev=cud, dq=dq, dk=dk, dv=dv)
    grad = ref.delta_bwd(host(do), *map(host, x.values()), host(init), host(dfinal), cu, n ** -0.5)
    for name, g, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dinit"), got, grad):
        assert rel(host(g), w) <= (BAR[dtype] if name in ("dq", "dk", "dv") else STATE[dtype]), name
    assert torch.all(grads[:, :8] == 7.0)           # columns beside them are left as they were
    assert torch.equal(got[5][0], dfinal[0])


@pytest.mark.parametrize("p,n,dtype", [(128, 128, "bf16"), (64, 64, "bf16"), (64, 64, "f32")])
def test_decays_of_all_sizes(p, n, dtype):
    """No decay, strong decay, a full reset (-infinity), and growth, side by side and in turn."""
    x, init, do, dfinal = inputs(11, 200, 1, 1, 4, p, n, dtype)
    g = x["g"]
    g[:, 0] = 0.0
    g[:, 1] = -3.0
    g[50:, 2] = 0.01
    g[70, 3] = g[128, 3] = g[0, 2] = float("-inf")
    g[100, 3] = -150.0
    o, final, kept = ssd.delta_scan_fwd(*batched(x, 1).values(), init, return_checkpoints=True)
    want, last, _ = ref.delta_fwd(*map(host, x.values()), host(init), [0, 200], n ** -0.5)
    got = ssd.delta_scan_bwd(do[None], *batched(x, 1).values(), kept, dfinal)
    grad = ref.delta_bwd(host(do), *map(host, x.values()), host(init), host(dfinal), [0, 200], n ** -0.5)
    for h in range(4):
        assert rel(host(o)[0, :, h], want[:, h]) <= BAR[dtype] and rel(host(final)[0, h], last[0, h]) <= STATE[dtype]
        for i in (2, 3, 4):
            assert rel(host(got[i])[0, :, h], grad[i][:, h]) <= (BAR[dtype] if i == 2 else STATE[dtype])
        if grad[5][0, h].any():
            assert rel(host(got[5])[0, h], grad[5][0, h]) <= STATE[dtype]
    assert torch.all(got[5][0, 2] == 0)


def test_without_states():
    x, _, do, _ = inputs(12, 100, 1, 1, 2, 64, 64, "bf16")
    b = batched(x, 1)
    zeros = torch.zeros((1, 2, 64, 64), device="cuda")
    o, none = ssd.delta_scan_fwd(*b.values(), return_final=False)
    assert none is None
    o2, final, kept = ssd.delta_scan_fwd(*b.values(), zeros, return_checkpoints=True)
    assert torch.equal(o, o2)
    got = ssd.delta_scan_bwd(do[None], *b.values(), kept, return_dinit=False)
    assert got[5] is None
    for a, c in zip(got[:5], ssd.delta_scan_bwd(do[None], *b.values(), kept, zeros)):
        assert torch.equal(a, c)


def test_tokens_that_write_nothing():
    """beta 0 (padding by value): the state passes, and what would be written has a gradient."""
    x, init, do, dfinal = inputs(17, 140, 1, 1, 2, 64, 128, "bf16")
    x["beta"][20:40] = 0.0
    x["beta"][139] = 0.0
    x["beta"][60, 0] = 1e-30
    o, final, kept = ssd.delta_scan_fwd(*batched(x, 1).values(), init, return_checkpoints=True)
    got = ssd.delta_scan_bwd(do[None], *batched(x, 1).values(), kept, dfinal)
    want, last, _ = ref.delta_fwd(*map(host, x.values()), host(init), [0, 140], 128 ** -0.5)
    grad = ref.delta_bwd(host(do), *map(host, x.values()), host(init), host(dfinal), [0, 140], 128 ** -0.5)
    assert rel(host(o)[0], want) <= BAR["bf16"] and rel(host(final), last) <= STATE["bf16"]
    for name, g, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dinit"), got, grad):
        assert rel(host(g).reshape(w.shape), w) <= (BAR["bf16"] if name in ("dq", "dk", "dv") else STATE["bf16"]), name
    assert rel(host(got[4])[0, 20:40], grad[4][20:40]) <= STATE["bf16"]


def test_what_lies_behind_a_sequence_stays_there():
    """NaN in the next sequence's tokens reaches nothing of this one."""
    cu = [0, 70, 140]
    x, init, do, dfinal = inputs(18, 140, 2, 1, 2, 128, 128, "bf16")
    clean = ssd.delta_scan_fwd(*x.values(), init, cu_seqlens=cu, return_checkpoints=True)
    grads = ssd.delta_scan_bwd(do, *x.values(), clean[2], dfinal, cu_seqlens=cu)
    for t in (*x.values(), do):
        t[70:] = float("nan")
    o, final, kept = ssd.delta_scan_fwd(*x.values(), init, cu_seqlens=cu, return_checkpoints=True)
    assert torch.equal(o[:70], clean[0][:70]) and torch.equal(final[0], clean[1][0]) and torch.isnan(final[1]).all()
    got = ssd.delta_scan_bwd(do, *x.values(), clean[2], dfinal, cu_seqlens=cu)
    for g, w in zip(got[:5], grads):
        assert torch.equal(g[:70], w[:70])
    assert torch.equal(got[5][0], grads[5][0])


@pytest.mark.parametrize("p,n", [(128, 128), (64, 64)])
def test_any_alignment(p, n):
    """Arrays that begin at any multiple of their element's size, and rows at odd strides."""
    x, init, do, dfinal = inputs(19, 70, 1, 1, 2, p, n, "bf16")
    b = batched(x, 1)
    want = ssd.delta_scan_fwd(*b.values(), init, return_checkpoints=True)
    grads = ssd.delta_scan_bwd(do[None], *b.values(), want[2], dfinal)

    def shifted(t):
        buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
        buf[1:] = t.reshape(-1)
        return buf[1:].view(t.shape)
    close = lambda got, ref_, bar: rel(host(got), host(ref_)) <= bar   # noqa: E731
    for which in (*b, "init", "o", "final_state", "checkpoints"):
        args = {name: shifted(t) if name == which else t for name, t in b.items()}
        out = {name: shifted(torch.zeros_like(t)) for name, t in (("o", want[0]), ("final_state", want[1]), ("checkpoints", want[2])) if name == which}
        got = ssd.delta_scan_fwd(*args.values(), shifted(init) if which == "init" else init, return_checkpoints=True, **out)
        assert close(got[0], want[0], 2 * BAR["bf16"]) and close(got[1], want[1], 2 * STATE["bf16"])
        assert close(got[2][:2], want[2][:2], 2 * STATE["bf16"]), which
    names = ("dq", "dk", "dv", "dg", "dbeta", "dinit")
    for which in (*b, "do", "kept", "dfinal", *names):
        args = {name: shifted(t) if name == which else t for name, t in b.items()}
        out = {which: shifted(torch.zeros_like(grads[names.index(which)]))} if which in names else {}
        got = ssd.delta_scan_bwd(shifted(do[None]) if which == "do" else do[None], *args.values(), shifted(want[2]) if which == "kept" else want[2],
                                 shifted(dfinal) if which == "dfinal" else dfinal, **out)
        for name, g, w in zip(names, got, grads):
            assert close(g, w, 2 * BAR["bf16"] if name in ("dq", "dk", "dv") else 2 * STATE["bf16"]), (which, name)
    wide = torch.zeros((1, 70, 2 * p + 3), dtype=torch.bfloat16, device="cuda")
    v = wide[..., 1:1 + 2 * p].unflatten(-1, (2, p))
    v.copy_(b["v"])
    o = torch.zeros_like(wide)[..., 2:2 + 2 * p].unflatten(-1, (2, p))
    assert close(ssd.delta_scan_fwd(**dict(b, v=v), o=o)[0], ssd.delta_scan_fwd(*b.values())[0], 2 * BAR["bf16"])


def test_the_first_part_then_the_rest():
    """A sequence cut in two gives what it gives whole: states are handed on in 32 bits."""
    x, init, _, _ = inputs(13, 320, 1, 2, 4, 128, 128, "bf16")
    whole, final = ssd.delta_scan_fwd(*batched(x, 1).values(), init)
    first, state = ssd.delta_scan_fwd(*(t[None, :192] for t in x.values()), init)
    rest, last = ssd.delta_scan_fwd(*(t[None, 192:] for t in x.values()), state)
    assert torch.equal(torch.cat([first, rest], 1), whole) and torch.equal(last, final)
    state = state.clone()
    for t in range(192, 200):
        o = ssd.delta_state_update(state, *(v[t:t + 1] for v in x.values()))
        assert rel(host(o[0]), host(whole[0, t])) <= 2 * BAR["bf16"]


STEP_SHAPES = [(1, 1, 1, 1, 1), (3, 1, 2, 5, 7), (16, 2, 4, 64, 128), (2, 2, 2, 128, 128), (5, 1, 3, 130, 20), (1, 1, 1, 33, 256), (4, 1, 2, 64, 64)]


@pytest.mark.parametrize("batch,groups,heads,p,n", STEP_SHAPES)
@pytest.mark.parametrize("dtype,sd", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16")])
def test_one_token(batch, groups, heads, p, n, dtype, sd):
    x, init, _, _ = inputs(p + n, batch, batch, groups, heads, p, n, dtype)
    state = init.to(DT[sd])
    old = state.clone()
    x["g"][0, 0] = float("-inf")
    want, last, _ = ref.delta_fwd(*map(host, x.values()), host(state), list(range(batch + 1)), 0.7)
    nxt = torch.full_like(state, float("nan"))
    o = ssd.delta_state_update(state, *x.values(), scale=0.7, state_out=nxt)
    assert torch.equal(state, old) and o.shape == (batch, heads, p) and o.dtype == DT[dtype]
    assert rel(host(o), want) <= BAR[dtype] and rel(host(nxt), last) <= BAR[sd]
    wide = torch.zeros((batch, 2 * groups * n + 3), dtype=DT[dtype], device="cuda")       # rows of a wider matrix
    q = wide[:, 1:1 + groups * n].unflatten(-1, (groups, n))
    q.copy_(x["q"])
    o2 = ssd.delta_state_update(state, **dict(x, q=q), scale=0.7, o=torch.empty_like(o))
    assert torch.equal(o2, o) and torch.equal(state, nxt)


def test_streams_and_graphs():
    x, init, do, dfinal = inputs(14, 150, 1, 1, 2, 128, 128, "bf16")
    b = batched(x, 1)

    def run(v):
        o, final, kept = ssd.delta_scan_fwd(b["q"], b["k"], v, b["g"], b["beta"], init, return_checkpoints=True)
        return (o, final) + ssd.delta_scan_bwd(do[None], b["q"], b["k"], v, b["g"], b["beta"], kept, dfinal)
    want = [t.clone() for t in run(b["v"])]
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        got = run(b["v"] * 1)
    side.synchronize()
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = run(b["v"])
    for _ in range(2):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(g, w) for g, w in zip(out, want))


def test_a_model_of_the_operators():
    """Tokens through the embedding, the layer norm, the products and the delta rule and
    back: gradients against torch's own of the same formulas in 64 bits, the weights as
    bf16 values.  Every bf16 tensor between two operators is rounded once (2^-9 of a value
    at random), some ten of them in a row: 3e-2."""
    rng = np.random.default_rng(15)
    vocab, width, groups, heads, p, n, batch, length = 50, 64, 1, 2, 32, 32, 2, 70
    table, norm_w, norm_b = dev(rng.standard_normal((vocab, width)), "bf16"), dev(1 + 0.1 * rng.standard_normal(width)), dev(0.1 * rng.standard_normal(width))
    w_in = dev(rng.standard_normal((2 * groups * n + heads * p, width)) * width ** -0.5, "bf16")
    w_out = dev(rng.standard_normal((width, heads * p)) * (heads * p) ** -0.5, "bf16")
    tokens = torch.from_numpy(rng.integers(0, vocab, (batch, length))).cuda()
    g, beta = dev(-0.2 * rng.random((batch, length, heads))), dev(0.2 * rng.random((batch, length, heads)))
    dout = dev(rng.standard_normal((batch, length, width)), "bf16")

    stream = ssd.embedding_fwd(tokens, table, scale=2.0, out_dtype=torch.float32)
    normed, _, mean, rstd, _ = ssd.layernorm_fwd(stream, norm_w, norm_b, out_dtype=torch.bfloat16)
    parts = ssd.linear_fwd(normed, w_in)
    cut = lambda m: (m[..., :n].unflatten(-1, (groups, n)), m[..., n:2 * n].unflatten(-1, (groups, n)),   # noqa: E731
                     m[..., 2 * n:].unflatten(-1, (heads, p)))
    q, k, v = cut(parts)
    o, _, kept = ssd.delta_scan_fwd(q, k, v, g, beta, scale=0.1, return_checkpoints=True)
    out = ssd.linear_fwd(o.flatten(-2), w_out, residual=stream, out_dtype=torch.float32)
    do, dw_out, _ = ssd.linear_bwd(dout, o.flatten(-2), w_out, bias=False)
    dparts = torch.empty_like(parts)
    dq, dk, dv = cut(dparts)
    _, _, _, dg, dbeta, _ = ssd.delta_scan_bwd(do.unflatten(-1, (heads, p)), q, k, v, g, beta, kept, scale=0.1, dq=dq, dk=dk, dv=dv)
    dnormed, dw_in, _ = ssd.linear_bwd(dparts, normed, w_in, bias=False)
    _, dstream, dnorm_w, dnorm_b = ssd.layernorm_bwd(dnormed, stream, norm_w, mean, rstd, dout.float())
    dtable = ssd.embedding_bwd(dstream, tokens, vocab, scale=2.0)

    leaves = [t.double().requires_grad_() for t in (table, norm_w, norm_b, w_in, w_out, g, beta)]
    ta, nw, nb, wi, wo, g6, b6 = leaves
    s6 = ta[tokens] * 2.0
    away = s6 - s6.mean(-1, keepdim=True)
    n6 = away * torch.rsqrt((away * away).mean(-1, keepdim=True) + 1e-5) * nw + nb
    q6, k6, v6 = cut(n6 @ wi.t())
    state, outs = torch.zeros((batch, heads, p, n), dtype=torch.float64, device="cuda"), []
    for t in range(length):
        kt, qt = k6[:, t].expand(-1, heads, -1), q6[:, t].expand(-1, heads, -1)
        state = torch.exp(g6[:, t])[..., None, None] * state
        u = b6[:, t][..., None] * (v6[:, t] - (state * kt[:, :, None]).sum(-1))
        state = state + u[..., None] * kt[:, :, None]
        outs.append(0.1 * (state * qt[:, :, None]).sum(-1))
    out6 = s6 + torch.stack(outs, 1).flatten(-2) @ wo.t()
    out6.backward(dout.double())
    assert rel(host(out), out6.detach().cpu().numpy()) <= 3e-2
    for name, got, leaf in zip(("table", "norm weight", "norm bias", "w_in", "w_out", "g", "beta"),
                               (dtable, dnorm_w, dnorm_b, dw_in, dw_out, dg, dbeta), leaves):
        assert rel(host(got), leaf.grad.cpu().numpy()) <= 3e-2, name


def test_refusals():
    x, init, do, _ = inputs(16, 8, 2, 2, 4, 16, 32, "bf16")
    b = batched(x, 2)
    q, k, v, g, beta = b.values()
    kept = torch.zeros((2, 4, 16, 32), device="cuda")
    for bad in (lambda: ssd.delta_scan_fwd(*x.values()),                         # tokens without offsets
                lambda: ssd.delta_scan_fwd(q.cpu(), k, v, g, beta), lambda: ssd.delta_scan_fwd(q, k[..., :16], v, g, beta),
                lambda: ssd.delta_scan_fwd(q, k, v[:, :3], g, beta), lambda: ssd.delta_scan_fwd(q, k, v, g[..., :2], beta),
                lambda: ssd.delta_scan_fwd(q, k, v, g, beta, init[:1]), lambda: ssd.delta_scan_fwd(q.transpose(-1, -2).contiguous().transpose(-1, -2), k, v, g, beta),
                lambda: ssd.delta_scan_fwd(*x.values(), cu_seqlens=[0, 9]), lambda: ssd.delta_scan_bwd(do.unflatten(0, (2, -1)), q, k, v, g, beta, None),
                lambda: ssd.delta_scan_bwd(do.unflatten(0, (2, -1)), q, k, v, g, beta, kept[:1]),
                lambda: ssd.delta_state_update(init[:, :, :8], x["q"][:2], x["k"][:2], x["v"][:2], x["g"][:2], x["beta"][:2]),
                lambda: ssd.delta_state_update(None, x["q"][:2], x["k"][:2], x["v"][:2], x["g"][:2], x["beta"][:2])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ssd.delta_scan_fwd(q, k, v.float(), g, beta), lambda: ssd.delta_scan_fwd(q, k, v, g.bfloat16(), beta)):
        with pytest.raises(TypeError):
            bad()
    three = torch.zeros((2, 4, 3, 32), dtype=torch.bfloat16, device="cuda")
    for bad in (lambda: ssd.delta_scan_fwd(three, three, v, g, beta),            # 4 heads in 3 groups
                lambda: ssd.delta_scan_fwd(*x.values(), cu_seqlens=[0, 5, 3, 8]),
                lambda: ssd.delta_scan_fwd(q, k, v, g, beta, scale=float("nan")),
                lambda: ssd.delta_state_update(init.bfloat16(), *(x[i][:2].float() for i in x))):
        with pytest.raises(ssd.SsdError):
            bad()


@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_short_and_long_way_of_a_call_agree(packed, dtype):
    """Calls that leave everything to be allocated go through compiled marshalling, others
    through Python: equal bits, with column ranges of one matrix and an outer dimension of one."""
    groups, heads, p, n = 2, 4, 64, 32
    lead = (150,) if packed else (3, 50)
    x, init, do, dfinal = inputs(21, 150, 3, groups, heads, p, n, dtype)
    wide = torch.zeros((*lead, 2 * groups * n + heads * p), dtype=DT[dtype], device="cuda")
    cuts = {"q": wide[..., :groups * n].unflatten(-1, (groups, n)),
            "k": wide[..., groups * n:2 * groups * n].unflatten(-1, (groups, n)),
            "v": wide[..., 2 * groups * n:].unflatten(-1, (heads, p))}
    for name, t in cuts.items():
        t.copy_(x[name].view(t.shape))
        x[name] = t
    for name in ("g", "beta"):
        x[name] = x[name].view(*lead, heads)
    do = do.view(*lead, heads, p)
    cu = [0, 20, 20, 150] if packed else None
    cud = torch.tensor(cu, dtype=torch.int32, device="cuda") if packed else None
    kw = dict(cu_seqlens=cu, cu_seqlens_dev=cud)
    short = ssd.delta_scan_fwd(*x.values(), init, scale=0.5, return_checkpoints=True, **kw)
    o = torch.empty_like(short[0])
    long = ssd.delta_scan_fwd(*x.values(), init, scale=0.5, return_checkpoints=True, o=o, **kw)
    assert long[0] is o and torch.equal(o, short[0]) and torch.equal(short[1], long[1])
    assert ssd.delta_scan_fwd(*x.values(), None, return_final=False, **kw)[1] is None
    back = ssd.delta_scan_bwd(do, *x.values(), short[2], dfinal, scale=0.5, **kw)
    dq = torch.empty_like(back[0])
    others = ssd.delta_scan_bwd(do, *x.values(), short[2], dfinal, scale=0.5, dq=dq, **kw)
    assert others[0] is dq and all(torch.equal(a, b) for a, b in zip(back, others))
    assert ssd.delta_scan_bwd(do, *x.values(), short[2], return_dinit=False, **kw)[5] is None
