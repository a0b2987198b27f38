"""The embedding on the GPU against tests/model_ref.py.  Bars as relative L2, derived
before the first run: bf16 outputs are rounded once (2^-8 of a value), f32 ones carry one
product (forward) or fp32 sums of up to some 10^4 rows (gradient): 4e-3 and 1e-5."""
import numpy as np
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import model_ref as ref
from tests.gpu_util import host, rel

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16}
BAR = {"f32": 1e-5, "bf16": 4e-3}


def tens(rng, shape, dtype="f32"):
    return torch.from_numpy(rng.standard_normal(shape).astype(np.float32)).to(DT[dtype]).cuda()


def ids(rng, shape, vocab, kind="spread", dtype=torch.int64):
    if kind == "spread":
        t = rng.integers(-1, vocab + 1, shape)              # also outside, on both sides
    elif kind == "one":
        t = np.full(shape, vocab // 2)
    elif kind == "none":
        t = np.full(shape, -1)
    else:                                                   # a few frequent ones
        t = np.minimum((vocab * rng.random(shape) ** 6).astype(np.int64), vocab - 1)
    return torch.from_numpy(np.asarray(t)).to(dtype).cuda()


@pytest.mark.parametrize("shape,vocab,width", [((1,), 1, 1), ((16, 1), 1000, 2560), ((3, 5, 2), 7, 33), ((700,), 300, 1024),
                                               ((2, 1031), 50, 72), ((9,), 11, 8200)])
@pytest.mark.parametrize("td,od", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("dtype", [torch.int32, torch.int64])
def test_lookup(shape, vocab, width, td, od, dtype):
    rng = np.random.default_rng(width)
    t, table = ids(rng, shape, vocab, dtype=dtype), tens(rng, (vocab, width), td)
    y = ssd.embedding_fwd(t, table, scale=3.0, out_dtype=DT[od])
    want = ref.embedding_fwd(t.cpu().numpy(), host(table), 3.0)
    assert y.shape == shape + (width,) and y.dtype == DT[od]
    assert rel(host(y), want) <= BAR[od] if want.any() else not host(y).any()


def test_lookup_without_scale_is_exact():
    rng = np.random.default_rng(2)
    t, table = ids(rng, (50,), 20, "few"), tens(rng, (20, 64), "bf16")
    assert torch.equal(ssd.embedding_fwd(t, table), table[t])


@pytest.mark.parametrize("shape,vocab,width,kind", [((1,), 1, 1, "spread"), ((3, 5), 7, 33, "spread"), ((31,), 5, 64, "one"),
                                                    ((33,), 5, 64, "one"), ((64,), 3, 1032, "spread"), ((5000,), 300, 264, "few"),
                                                    ((4, 1031), 600, 40, "spread"), ((9000,), 70000, 16, "few"),
                                                    ((2049,), 9, 100, "one"), ((70,), 513, 8, "none"), ((40000,), 250001, 8, "spread"),
                                                    ((90000,), 3000, 8, "few"), ((90001,), 300000, 4, "spread"), ((2000,), 30000, 640, "few")])
@pytest.mark.parametrize("d,od", [("f32", "f32"), ("bf16", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
def test_gradient(shape, vocab, width, kind, d, od):
    rng = np.random.default_rng(vocab + width)
    t, dy = ids(rng, shape, vocab, kind), tens(rng, shape + (width,), d)
    out = torch.full((vocab, width), float("nan"), dtype=DT[od], device="cuda")
    got = ssd.embedding_bwd(dy, t, vocab, scale=0.5, dtype=DT[od], dtable=out)
    assert got is out
    want = ref.embedding_bwd(host(dy), t.cpu().numpy(), vocab, 0.5)
    got = host(got)
    assert np.all(got[~np.isin(np.arange(vocab), t.cpu().numpy())] == 0)
    assert rel(got, want) <= BAR[od] if want.any() else not got.any()


def test_gradient_is_the_same_every_time_and_follows_strides():
    rng = np.random.default_rng(8)
    t = ids(rng, (3, 4000), 1000, "few", torch.int32)
    wide = tens(rng, (3, 4000, 96), "bf16")
    dy = wide[..., 16:80]
    first = ssd.embedding_bwd(dy, t, 1000)
    want = ref.embedding_bwd(host(dy), t.cpu().numpy(), 1000, 1.0)
    assert first.dtype == torch.bfloat16 and rel(host(first), want) <= BAR["bf16"]
    for _ in range(3):
        assert torch.equal(ssd.embedding_bwd(dy, t, 1000), first)
    assert torch.equal(ssd.embedding_bwd(wide[..., 15:79], t, 1000), ssd.embedding_bwd(wide[..., 15:79].contiguous(), t, 1000))


def test_rows_of_nan_reach_only_their_token():
    rng = np.random.default_rng(9)
    t, dy = ids(rng, (100,), 10, "spread"), tens(rng, (100, 64))
    t[5], t[6] = 3, -1
    dy[5] = float("nan")
    dy[6] = float("inf")        # of a padding token
    got = ssd.embedding_bwd(dy, t, 10)
    assert torch.isnan(got[3]).all() and torch.isfinite(got[[0, 1, 2, 4, 5, 6, 7, 8, 9]]).all()
    table = tens(rng, (10, 64))
    table[0] = float("nan")     # nor does the first row reach a padding token
    assert torch.all(ssd.embedding_fwd(torch.tensor([-1, 10], device="cuda"), table) == 0)


def test_empty_calls():
    t, table = torch.zeros((0, 4), dtype=torch.int64, device="cuda"), torch.zeros((5, 8), device="cuda")
    y = ssd.embedding_fwd(t, table)
    assert y.shape == (0, 4, 8)
    assert torch.all(ssd.embedding_bwd(y, t, 5, dtable=torch.ones((5, 8), device="cuda")) == 0)


def test_streams_and_graphs():
    rng = np.random.default_rng(10)
    t, dy = ids(rng, (3000,), 500, "few"), tens(rng, (3000, 128), "bf16")
    want = ssd.embedding_bwd(dy, t, 500, dtype=torch.float32)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)
        got = ssd.embedding_bwd(dy * 2, t, 500, dtype=torch.float32)
    side.synchronize()
    assert torch.equal(got, want * 2)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = ssd.embedding_bwd(dy, t, 500, dtype=torch.float32)
    for _ in range(2):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    t.copy_(ids(rng, (3000,), 500, "spread"))           # other tokens, the same graph
    graph.replay()
    torch.cuda.synchronize()
    assert rel(host(out), ref.embedding_bwd(host(dy), t.cpu().numpy(), 500, 1.0)) <= BAR["f32"]


def test_refusals():
    t, table = torch.zeros((4,), dtype=torch.int64, device="cuda"), torch.zeros((5, 8), device="cuda")
    dy = torch.zeros((4, 8), device="cuda")
    for bad in (lambda: ssd.embedding_fwd(t.cpu(), table), lambda: ssd.embedding_fwd(t, table[0]),
                lambda: ssd.embedding_fwd(t, table[:, :4]), lambda: ssd.embedding_fwd(t.repeat(2)[::2], table),
                lambda: ssd.embedding_bwd(dy[:3], t, 5), lambda: ssd.embedding_bwd(dy, t, 0),
                lambda: ssd.embedding_bwd(dy, t, 5, dtable=table[:4])):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ssd.embedding_fwd(t.float(), table), lambda: ssd.embedding_fwd(t, table.double()),
                lambda: ssd.embedding_bwd(dy.half(), t, 5)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ssd.embedding_fwd(t, table, scale=float("inf")), lambda: ssd.embedding_fwd(t, table.to(torch.float8_e4m3fn)),
                lambda: ssd.embedding_bwd(dy, t, 5, scale=float("nan"))):
        with pytest.raises(ssd.SsdError):
            bad()
