"""Which kernels the delta rule's calls take, by choice.  With bf16 inputs the fp32 kernels'
f32 results are within 1e-6 (fp32 sums along a memory of some 10^2 tokens, each step off by
2^-24 = 6e-8 of the state at random), where the tensor cores' are held to 3e-5
(test_delta_gpu.py)."""
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import model_ref as ref
from tests.gpu_util import host, rel
from tests.test_delta_gpu import BAR, inputs

pytestmark = pytest.mark.gpu

UNSUPPORTED = 2     # SSD_ERR_UNSUPPORTED
FINE = 1e-6


def shifted(t):
    buf = torch.zeros(t.numel() + 1, dtype=t.dtype, device="cuda")
    buf[1:] = t.reshape(-1)
    return buf[1:].view(t.shape)


@pytest.mark.parametrize("cu,groups,heads,p,n", [([0, 200], 1, 2, 64, 128), ([0, 70, 70, 300], 2, 4, 128, 64), ([0, 1700], 1, 1, 64, 64)])
def test_the_fp32_kernels_by_choice(cu, groups, heads, p, n):
    x, init, do, dfinal = inputs(n, cu[-1], len(cu) - 1, groups, heads, p, n, "bf16")
    kw = dict(cu_seqlens=cu, algo=ssd.ALGO_SIMT)
    o, final, kept = ssd.delta_scan_fwd(*x.values(), init, return_checkpoints=True, **kw)
    got = ssd.delta_scan_bwd(do, *x.values(), kept, dfinal, **kw)
    want, last, before = ref.delta_fwd(*map(host, x.values()), host(init), cu, n ** -0.5)
    grad = ref.delta_bwd(host(do), *map(host, x.values()), host(init), host(dfinal), cu, n ** -0.5)
    assert rel(host(o), want) <= BAR["bf16"] and rel(host(final), last) <= FINE
    for place, state in ref.delta_kept(before, cu):
        assert rel(host(kept[place]), state) <= FINE
    for name, g, w in zip(("dq", "dk", "dv", "dg", "dbeta", "dinit"), got, grad):
        assert rel(host(g), w) <= (BAR["bf16"] if g.dtype == torch.bfloat16 else 10 * FINE if name in ("dg", "dbeta") else FINE), name
    # what an address that the tensor cores do not take gets without asking: the same bits
    odd = dict(x, q=shifted(x["q"]))
    o2, final2, kept2 = ssd.delta_scan_fwd(*odd.values(), init, cu_seqlens=cu, return_checkpoints=True)
    assert torch.equal(o, o2) and torch.equal(final, final2)
    assert all(torch.equal(a, b) for a, b in zip(got, ssd.delta_scan_bwd(do, *odd.values(), kept, dfinal, cu_seqlens=cu)))


def test_the_tensor_cores_by_choice():
    x, init, do, dfinal = inputs(3, 150, 1, 1, 2, 64, 64, "bf16")
    b = {name: t[None] for name, t in x.items()}
    plain = ssd.delta_scan_fwd(*b.values(), init, return_checkpoints=True)
    asked = ssd.delta_scan_fwd(*b.values(), init, return_checkpoints=True, algo=ssd.ALGO_TCGEN05)
    assert torch.equal(plain[0], asked[0]) and torch.equal(plain[1], asked[1])
    grads = ssd.delta_scan_bwd(do[None], *b.values(), plain[2], dfinal)
    assert all(torch.equal(g, w) for g, w in zip(ssd.delta_scan_bwd(do[None], *b.values(), plain[2], dfinal, algo=ssd.ALGO_TCGEN05), grads))
    # checkpoints of either choice
    fine = ssd.delta_scan_fwd(*b.values(), init, return_checkpoints=True, algo=ssd.ALGO_SIMT)
    mixed = ssd.delta_scan_bwd(do[None], *b.values(), fine[2], dfinal)
    assert all(rel(host(g), host(w)) <= (2 * BAR["bf16"] if g.dtype == torch.bfloat16 else 6e-5) for g, w in zip(mixed, grads))


def test_choices_refused():
    x, init, do, _ = inputs(4, 20, 1, 1, 2, 64, 64, "bf16")
    b = {name: t[None] for name, t in x.items()}
    kept = torch.zeros((1, 2, 64, 64), device="cuda")
    odd, wide = {name: t[None] for name, t in inputs(4, 20, 1, 1, 2, 60, 64, "bf16")[0].items()}, inputs(4, 20, 1, 1, 2, 136, 64, "bf16")
    full = {name: t[None] for name, t in inputs(4, 20, 1, 1, 2, 64, 64, "f32")[0].items()}
    kw = dict(algo=ssd.ALGO_TCGEN05)
    for bad in (lambda: ssd.delta_scan_fwd(*odd.values(), **kw), lambda: ssd.delta_scan_fwd(*full.values(), **kw),
                lambda: ssd.delta_scan_fwd(*dict(b, k=shifted(b["k"])).values(), **kw),
                lambda: ssd.delta_scan_bwd(shifted(do[None]), *b.values(), kept, **kw),
                # forward blocks of 128 rows, gradients one
                lambda: ssd.delta_scan_bwd(wide[2][None], *(t[None] for t in wide[0].values()), torch.zeros((1, 2, 136, 64), device="cuda"), **kw)):
        with pytest.raises(ssd.SsdError) as e:
            bad()
        assert e.value.code == UNSUPPORTED
    for bad in (lambda: ssd.delta_scan_fwd(*b.values(), algo=3), lambda: ssd.delta_scan_bwd(do[None], *b.values(), kept, algo=-1)):
        with pytest.raises(ssd.SsdError):
            bad()


def test_no_tokens():
    q = torch.zeros((2, 0, 1, 64), dtype=torch.bfloat16, device="cuda")
    v, g, init = torch.zeros((2, 0, 2, 64), dtype=torch.bfloat16, device="cuda"), torch.zeros((2, 0, 2), device="cuda"), torch.randn((2, 2, 64, 64), device="cuda")
    for algo in (ssd.ALGO_AUTO, ssd.ALGO_SIMT, ssd.ALGO_TCGEN05):
        o, final = ssd.delta_scan_fwd(q, q, v, g, g, init, algo=algo)
        assert o.shape == v.shape and torch.equal(final, init)
