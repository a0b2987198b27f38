"""The layer norm on the GPU against tests/model_ref.py, on the inputs as the GPU holds
them.  Bars as relative L2, derived before the first run: bf16 outputs are rounded once,
by at most 2^-8 of a value (3.91e-3), with below 1e-5 in front: 4e-3; f32 outputs are sums
of up to 10^4 fp32 terms: 1e-5; 8-bit values half a step of E4M3, 2^-4 |y| plus 2^-10 of
the scale for subnormals (and 1e-5 for the fp32 in front, against the row's largest |y|,
since bias and normed value can cancel)."""
import numpy as np
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import model_ref as ref
from tests.gpu_util import host, rel

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
BAR = {"f32": 1e-5, "bf16": 4e-3}


def tens(rng, shape, dtype="f32", std=1.0, mean=0.0):
    a = (rng.standard_normal(shape) * std + mean).astype(np.float32)
    return torch.from_numpy(a).to(DT[dtype]).cuda()


def cols(rng, rows, width, pad, dtype, **kw):
    return tens(rng, (rows, width + pad), dtype, **kw)[:, pad // 2:pad // 2 + width]


SHAPES = [(1, 1), (3, 7), (5, 64), (200, 250), (1, 2560), (16, 2560), (333, 2560), (4, 4096), (3, 8184), (2, 8191),
          (2, 32768), (2, 33000), (700, 1024), (1, 264), (40, 1000)]


@pytest.mark.parametrize("rows,width", SHAPES)
@pytest.mark.parametrize("xd,rd,od,bias", [("bf16", None, "bf16", True), ("bf16", "bf16", "fp8", True),
                                           ("bf16", "f32", "bf16", False), ("bf16", "f32", "fp8", False),
                                           ("f32", "f32", "f32", True), ("f32", None, "fp8", True),
                                           ("bf16", "f32", "f32", True), ("f32", "f32", "bf16", False)])
def test_forward(rows, width, xd, rd, od, bias):
    rng = np.random.default_rng(rows * 7 + width)
    x, w = tens(rng, (rows, width), xd, mean=0.5), tens(rng, (width,), std=0.3, mean=1.0)
    b = tens(rng, (width,), std=0.5) if bias else None
    r = tens(rng, (rows, width), rd, std=3.0, mean=2.0) if rd else None
    y, s, mean, rstd, scale = ssd.layernorm_fwd(x, w, b, r, eps=1e-5, out_dtype=DT[od])
    yr, sr, mr, rr = ref.layernorm_fwd(host(x), None if r is None else host(r), host(w), None if b is None else host(b), 1e-5)
    # a mean's error is held against its row's size
    assert np.linalg.norm(host(mean) - mr) <= BAR["f32"] * np.linalg.norm(np.sqrt((sr * sr).mean(axis=-1)))
    if width > 1:
        assert rel(host(rstd), rr) <= BAR["f32"]
    if r is None:
        assert s is None
    else:
        assert s.dtype == r.dtype and rel(host(s), sr) <= BAR[rd]
    if width == 1:      # one value is its own mean: y is the bias
        assert np.allclose(host(y) * (host(scale)[:, None] if od == "fp8" else 1.0), 0.0 if b is None else host(b), rtol=2.0 ** -4, atol=1e-3)
        return
    if od != "fp8":
        assert y.dtype == DT[od] and scale is None and rel(host(y), yr) <= BAR[od]
        return
    top = np.abs(yr).max(axis=-1)
    assert rel(host(scale), top / 448.0) <= BAR["f32"]
    sc = host(scale)[:, None]
    assert np.all(np.abs(host(y) * sc - yr) <= np.abs(yr) * 2.0 ** -4 + 1e-5 * top[:, None] + sc * 2.0 ** -10)
    assert np.all(np.abs(host(y)).max(axis=-1) == 448.0)


@pytest.mark.parametrize("width", [96, 97, 2048])
def test_large_means_and_far_values(width):
    """Rows whose mean is 10^3 times their spread, and rows with one far value first."""
    rng = np.random.default_rng(width)
    x = tens(rng, (7, width), "f32", mean=1000.0)
    x[3:] -= 1000.0
    x[3:, 0] = 3000.0
    w = tens(rng, (width,))
    y, _, mean, rstd, _ = ssd.layernorm_fwd(x, w)
    yr, _, mr, rr = ref.layernorm_fwd(host(x), None, host(w), None, 1e-5)
    # a value's distance from the mean is known to the mean's last bit: 2^-24 * 1000 of a spread of 1
    assert np.all(np.abs(host(mean) - mr) <= 2e-7 * np.sqrt((host(x) ** 2).mean(axis=-1)))
    assert np.all(np.abs(host(rstd) - rr) <= 1e-5 * rr)
    assert rel(host(y[:3]), yr[:3]) <= 4e-4 and rel(host(y[3:]), yr[3:]) <= 1e-5


@pytest.mark.parametrize("width", [96, 97])
def test_strided_in_place_and_leading_dimensions(width):
    rng = np.random.default_rng(width)
    x = cols(rng, 12, width, 8, "bf16").unflatten(0, (3, 4))
    r, w = tens(rng, (3, 4, width), "f32"), tens(rng, (width,))
    yr, sr, _, _ = ref.layernorm_fwd(host(x), host(r), host(w), None, 1e-5)
    y, s, mean, rstd, _ = ssd.layernorm_fwd(x, w, None, r, residual_out=r)
    assert s is r and mean.shape == rstd.shape == (3, 4) and y.shape == (3, 4, width)
    assert rel(host(y), yr) <= BAR["bf16"] and rel(host(r), sr) <= BAR["f32"]


def test_constant_rows_infinities_and_nan_stay_in_their_rows():
    rng = np.random.default_rng(5)
    x, w, b = tens(rng, (6, 300), "f32"), tens(rng, (300,), std=0.3, mean=1.0), tens(rng, (300,))
    x[1] = 4.0
    x[2, 17] = float("nan")
    x[3, 5] = float("inf")
    clean = ref.layernorm_fwd(host(x[[0, 1, 4, 5]]), None, host(w), host(b), 1e-5)[0]
    for od in ("f32", "bf16"):
        y = ssd.layernorm_fwd(x, w, b, out_dtype=DT[od])[0]
        assert rel(host(y[[0, 1, 4, 5]]), clean) <= BAR[od]
        assert torch.isnan(y[2].float()).all() and torch.isnan(y[3].float()).all()
    y8, _, _, rstd, scale = ssd.layernorm_fwd(x, w, b, out_dtype=DT["fp8"])
    assert torch.isnan(scale[2]) and torch.isnan(y8[2].float()).all() and torch.isnan(rstd[3])
    y, _, _, _, scale = ssd.layernorm_fwd(x[1:2], w, out_dtype=DT["fp8"])       # a constant row without bias
    assert torch.all(y.float() == 0) and scale.item() == 1.0


@pytest.mark.parametrize("rows,width", SHAPES)
@pytest.mark.parametrize("d,sd,dres,bias", [("bf16", "bf16", True, True), ("bf16", "f32", True, False),
                                            ("bf16", "f32", False, True), ("f32", "f32", True, True)])
def test_backward(rows, width, d, sd, dres, bias):
    rng = np.random.default_rng(rows * 3 + width)
    s, w = tens(rng, (rows, width), sd, std=2.0, mean=1.0), tens(rng, (width,), std=0.3, mean=1.0)
    dy = cols(rng, rows, width, 16, d)
    dr = tens(rng, (rows, width), sd) if dres else None
    _, _, mr, rr = ref.layernorm_fwd(host(s), None, host(w), None, 1e-5)
    mean, rstd = (torch.from_numpy(t.astype(np.float32)).cuda() for t in (mr, rr))
    dx, ds, dw, db = ssd.layernorm_bwd(dy, s, w, mean, rstd, dr, bias=bias)
    dsr, dwr, dbr = ref.layernorm_bwd(host(dy), host(s), host(w), host(mean), host(rstd), host(dr) if dres else None)
    # where a row is a value or two, ds cancels: held against the terms' size
    size = np.linalg.norm(host(dy) * host(w) * host(rstd)[:, None]) + (np.linalg.norm(host(dr)) if dres else 0)
    err = lambda t: np.linalg.norm(host(t) - dsr) / size   # noqa: E731
    assert err(dx) <= BAR[d] and err(ds) <= BAR[sd]
    assert (ds is dx) == (d == sd) and (db is not None) == bias
    v = (host(s) - host(mean)[:, None]) * host(rstd)[:, None]
    assert np.linalg.norm(host(dw) - dwr) <= BAR["f32"] * max(np.linalg.norm(dwr), np.sqrt(((host(dy) * v) ** 2).sum()), 1e-30)
    if bias:
        assert np.linalg.norm(host(db) - dbr) <= BAR["f32"] * max(np.linalg.norm(dbr), np.linalg.norm(host(dy)))


def test_empty_calls():
    w = torch.ones(8, device="cuda")
    x = torch.zeros((0, 8), device="cuda")
    y, _, mean, rstd, _ = ssd.layernorm_fwd(x, w)
    assert y.shape == (0, 8) and mean.shape == rstd.shape == (0,)
    dx, _, dw, db = ssd.layernorm_bwd(x, x, w, mean, rstd, dweight=torch.ones_like(w), dbias=torch.ones_like(w))
    assert dx.shape == (0, 8) and torch.all(dw == 0) and torch.all(db == 0)


def test_refusals():
    bf = torch.bfloat16
    x, w = torch.zeros((4, 64), dtype=bf, device="cuda"), torch.zeros((64,), device="cuda")
    m = torch.zeros((4,), device="cuda")
    for bad in (lambda: ssd.layernorm_fwd(x.cpu(), w), lambda: ssd.layernorm_fwd(x, w[:32]),
                lambda: ssd.layernorm_fwd(x, w, w[:32]), lambda: ssd.layernorm_fwd(x.t(), m),
                lambda: ssd.layernorm_fwd(x, w, None, x[:2]), lambda: ssd.layernorm_bwd(x, x, w, m[:3], m),
                lambda: ssd.layernorm_bwd(x, x, w, m, m, bias=False, dbias=w), lambda: ssd.layernorm_fwd(x, w, residual_out=x)):
        with pytest.raises(ValueError):
            bad()
    for bad in (lambda: ssd.layernorm_fwd(x, w.to(bf)), lambda: ssd.layernorm_fwd(x.double(), w),
                lambda: ssd.layernorm_bwd(x, x, w, m.double(), m)):
        with pytest.raises(TypeError):
            bad()
    for bad in (lambda: ssd.layernorm_fwd(x, w, eps=-1.0), lambda: ssd.layernorm_fwd(x.float(), w, None, x),
                lambda: ssd.layernorm_fwd(x.to(DT["fp8"]), w)):
        with pytest.raises(ssd.SsdError):
            bad()


@pytest.mark.parametrize("rows,width", [(2431, 264), (2432, 8), (2432, 512), (2433, 776), (3000, 1024), (2440, 1544),
                                        (5003, 2048), (2600, 2560), (2450, 4096), (2450, 4104), (2450, 1001)])
@pytest.mark.parametrize("xd,rd,pad", [("bf16", None, 0), ("bf16", "bf16", 8), ("bf16", "f32", 0), ("f32", "f32", 4),
                                       ("f32", None, 2), ("bf16", "bf16", 2)])
def test_many_rows_to_8_bits(rows, width, xd, rd, pad):
    """Around the number of rows from which on a row is a warp's; rows whose addresses and
    strides rule that out among them (pad 2)."""
    rng = np.random.default_rng(rows + width)
    x, w = cols(rng, rows, width, pad, xd, mean=0.5), tens(rng, (width,), std=0.3, mean=1.0)
    b, r = tens(rng, (width,), std=0.5), cols(rng, rows, width, pad, rd, std=3.0) if rd else None
    y, s, mean, rstd, scale = ssd.layernorm_fwd(x, w, b, r, eps=1e-5, out_dtype=DT["fp8"])
    yr, sr, mr, rr = ref.layernorm_fwd(host(x), None if r is None else host(r), host(w), host(b), 1e-5)
    assert np.linalg.norm(host(mean) - mr) <= BAR["f32"] * np.linalg.norm(np.sqrt((sr * sr).mean(axis=-1)))
    assert rel(host(rstd), rr) <= BAR["f32"]
    assert s is None if r is None else rel(host(s), sr) <= BAR[rd]
    top, sc = np.abs(yr).max(axis=-1), host(scale)[:, None]
    assert rel(host(scale), top / 448.0) <= BAR["f32"]
    assert np.all(np.abs(host(y) * sc - yr) <= np.abs(yr) * 2.0 ** -4 + 1e-5 * top[:, None] + sc * 2.0 ** -10)
