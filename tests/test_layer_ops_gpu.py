"""The layer's steps around the scan on the GPU against the plain 64-bit
implementations of tests/layer_ref.py, on the inputs as the GPU holds them.

Bars, as relative L2 unless said otherwise, derived before the first run:
  bf16 outputs   each value is rounded once to 8 significant bits, by at most
                 2^-8 of itself (3.91e-3); the fp32 arithmetic in front adds
                 below 1e-5: 4e-3.
  bf16 dx, dw of a product with an activation: dp is rounded once more in front
                 of the products, independently value by value: twice that, 8e-3.
  f32 outputs    sums of up to 10^4 fp32 terms and the hardware's exponential
                 and reciprocal (a few 2^-23 each): 1e-5.  The recurrence
                 multiplies a gate's rounding (2^-24) along its memory of up to
                 ~10^3 tokens, which averages out below the same bar.
  8-bit outputs  value by value: half a step of E4M3, 2^-4 |y| plus 2^-10 of the
                 scale for subnormals (and 1e-5 for the fp32 in front).
"""
import numpy as np
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import layer_ref as ref
from tests.gpu_util import host, rel

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "bf16": torch.bfloat16, "fp8": torch.float8_e4m3fn}
BAR = {"f32": 1e-5, "bf16": 4e-3}


def tens(rng, shape, dtype="f32", std=1.0, mean=0.0):
    a = (rng.standard_normal(shape) * std + mean).astype(np.float32)
    return torch.from_numpy(a).to(DT[dtype]).cuda()


def cols(rng, rows, width, pad, dtype, **kw):
    """A column range of a wider matrix: [rows, width] with row stride width + pad."""
    return tens(rng, (rows, width + pad), dtype, **kw)[:, pad // 2:pad // 2 + width]


# ----------------------------------------------------------------------- norm
NORM_SHAPES = [(1, 1), (3, 7), (5, 64), (200, 250), (1, 2560), (16, 2560), (333, 2560), (4, 4096),
               (3, 8184), (2, 8191), (2, 32768), (2, 33000), (700, 1024)]


@pytest.mark.parametrize("rows,width", NORM_SHAPES)
@pytest.mark.parametrize("xd,rd,od", [("bf16", None, "bf16"), ("bf16", "bf16", "fp8"),
                                      ("bf16", "f32", "bf16"), ("bf16", "f32", "fp8"),
                                      ("f32", "f32", "f32"), ("f32", None, "fp8"),
                                      ("bf16", "f32", "f32"), ("f32", "f32", "bf16")])
def test_norm_fwd(rows, width, xd, rd, od):
    rng = np.random.default_rng(rows * 7 + width)
    x, w = tens(rng, (rows, width), xd), tens(rng, (width,), std=0.3, mean=1.0)
    r = tens(rng, (rows, width), rd, std=3.0) if rd else None
    y, s, rstd, scale = ssd.rmsnorm_fwd(x, w, r, eps=1e-5, out_dtype=DT[od])
    yr, sr, rr = ref.norm_fwd(host(x), None if r is None else host(r), host(w), 1e-5)
    assert rel(host(rstd), rr) <= BAR["f32"]
    if r is None:
        assert s is None
    else:
        assert s.dtype == r.dtype and rel(host(s), sr) <= BAR[rd]
    if od != "fp8":
        assert y.dtype == DT[od] and scale is None and rel(host(y), yr) <= BAR[od]
        return
    top = np.abs(yr).max(axis=-1)
    assert rel(host(scale), top / ref.E4M3_MAX) <= BAR["f32"]
    sc = host(scale)[:, None]
    got = host(y) * sc
    assert np.all(np.abs(got - yr) <= np.abs(yr) * (2.0 ** -4 + 1e-5) + sc * 2.0 ** -10)
    assert np.all(np.abs(host(y)).max(axis=-1) == ref.E4M3_MAX)


@pytest.mark.parametrize("width", [96, 97])
def test_norm_strided_in_place_and_leading_dimensions(width):
    rng = np.random.default_rng(width)
    x = cols(rng, 12, width, 8, "bf16").unflatten(0, (3, 4))
    r = tens(rng, (3, 4, width), "f32")
    w = tens(rng, (width,))
    yr, sr, _ = ref.norm_fwd(host(x), host(r), host(w), 1e-5)
    y, s, rstd, _ = ssd.rmsnorm_fwd(x, w, r, residual_out=r)
    assert s is r and rstd.shape == (3, 4) and y.shape == (3, 4, width)
    assert rel(host(y), yr) <= BAR["bf16"] and rel(host(r), sr) <= BAR["f32"]


def test_norm_rows_of_zeros_infinities_and_nan_stay_in_their_rows():
    rng = np.random.default_rng(5)
    x = tens(rng, (6, 300), "f32")
    x[1] = 0.0
    x[2, 17] = float("nan")
    x[3, 5] = float("inf")
    x[4] *= 1e-36
    w = tens(rng, (300,), std=0.3, mean=1.0)
    y, _, rstd, scale = ssd.rmsnorm_fwd(x, w, eps=0.0, out_dtype=DT["fp8"])
    y1, _, _, s1 = ssd.rmsnorm_fwd(x[1:2], w, eps=1e-5, out_dtype=DT["fp8"])
    assert torch.all(y1.float() == 0) and s1.item() == 1.0
    for row in (0, 5):
        yr = ref.norm_fwd(host(x[row:row + 1]), None, host(w), 0.0)[0]
        got = host(y[row:row + 1]) * host(scale[row:row + 1])[:, None]
        assert np.all(np.abs(got - yr) <= np.abs(yr) * (2.0 ** -4 + 1e-5) + host(scale)[row] * 2.0 ** -10)
    assert torch.isnan(rstd[2]) and torch.isnan(y[2].float()).all() and torch.isnan(scale[2])
    # an infinite value: rstd is 0, finite values give 0 and the infinite one NaN
    yf, _, rf, _ = ssd.rmsnorm_fwd(x[3:4], w)
    assert rf.item() == 0.0 and torch.isnan(yf[0, 5]) and torch.isnan(yf[0]).sum() == 1


@pytest.mark.parametrize("rows,width", NORM_SHAPES)
@pytest.mark.parametrize("d,sd,dres", [("bf16", "bf16", True), ("bf16", "f32", True),
                                       ("bf16", "f32", False), ("f32", "f32", True)])
def test_norm_bwd(rows, width, d, sd, dres):
    rng = np.random.default_rng(rows * 3 + width)
    s, w = tens(rng, (rows, width), sd, std=2.0), tens(rng, (width,), std=0.3, mean=1.0)
    dy = cols(rng, rows, width, 16, d)
    dr = tens(rng, (rows, width), sd) if dres else None
    rstd = torch.from_numpy((1 / np.sqrt((host(s) ** 2).mean(-1) + 1e-5)).astype(np.float32)).cuda()
    dx, ds, dw = ssd.rmsnorm_bwd(dy, s, w, rstd, dr)
    dsr, dwr = ref.norm_bwd(host(dy), host(s), host(w), host(rstd), host(dr) if dres else None)
    # where a row is one value, ds cancels to eps-sized remainders: held against the terms' size
    size = np.linalg.norm(host(dy) * host(w) * host(rstd)[:, None]) + (np.linalg.norm(host(dr)) if dres else 0)
    err = lambda t: np.linalg.norm(host(t) - dsr) / max(size, 1e-30)   # noqa: E731
    assert err(dx) <= BAR[d] and err(ds) <= BAR[sd]
    assert (ds is dx) == (d == sd)
    wsize = np.sqrt(((host(dy) * host(s) * host(rstd)[:, None]) ** 2).sum())
    assert np.linalg.norm(host(dw) - dwr) <= BAR["f32"] * max(wsize, np.linalg.norm(dwr))


# -------------------------------------------------------------------- product
PRODUCT_SHAPES = [(1, 1, 1), (1, 256, 128), (3, 5, 7), (17, 64, 40), (16, 640, 512), (64, 80, 2064),
                  (65, 48, 80), (128, 128, 64), (129, 272, 144), (300, 500, 96), (257, 1040, 1000),
                  (1000, 96, 33), (640, 24, 4096), (2500, 520, 264)]


@pytest.mark.parametrize("m,n,k", PRODUCT_SHAPES)
@pytest.mark.parametrize("d,od,act,bias,res", [("bf16", "bf16", "none", False, False),
                                               ("bf16", "bf16", "silu", True, True),
                                               ("bf16", "f32", "gelu", True, False),
                                               ("f32", "f32", "relu", True, True),
                                               ("f32", "f32", "none", False, True)])
def test_linear_fwd(m, n, k, d, od, act, bias, res):
    rng = np.random.default_rng(m + n * 3 + k)
    x, w = tens(rng, (m, k), d), tens(rng, (n, k), d, std=k ** -0.5)
    b = tens(rng, (n,)) if bias else None
    r = tens(rng, (m, n), od) if res else None
    y, p = ssd.linear_fwd(x, w, b, r, activation=act, out_dtype=DT[od], return_preact=True)
    yr, pr = ref.linear_fwd(host(x), host(w), host(b) if bias else None, host(r) if res else None, act)
    assert y.dtype == DT[od] and rel(host(y), yr) <= BAR[od]
    assert rel(host(p), pr) <= BAR["f32" if d == "f32" else "bf16"]
    y2 = ssd.linear_fwd(x, w, b, r, activation=act, out_dtype=DT[od])
    assert torch.equal(y, y2)


@pytest.mark.parametrize("m,n,k", [(1, 16, 16), (1, 512, 2048), (5, 30, 36), (16, 272, 5120),
                                   (100, 96, 48), (129, 256, 144), (700, 520, 272)])
@pytest.mark.parametrize("od,act,bias,res", [("bf16", "silu", True, False), ("f32", "none", False, True)])
def test_linear_fwd_8_bit(m, n, k, od, act, bias, res):
    rng = np.random.default_rng(m + n + k)
    xf, wf = tens(rng, (m, k)), tens(rng, (n, k), std=k ** -0.5)
    ones = torch.ones(k, device="cuda")
    x, _, _, xs = ssd.rmsnorm_fwd(xf, ones, out_dtype=DT["fp8"])
    w, _, _, ws = ssd.rmsnorm_fwd(wf, ones, out_dtype=DT["fp8"])
    b = tens(rng, (n,)) if bias else None
    r = tens(rng, (m, n), od) if res else None
    y = ssd.linear_fwd(x, w, b, r, activation=act, x_scale=xs, w_scale=ws, out_dtype=DT[od])
    yr, _ = ref.linear_fwd(host(x), host(w), host(b) if bias else None, host(r) if res else None, act,
                           host(xs), host(ws))
    assert rel(host(y), yr) <= BAR[od]


@pytest.mark.parametrize("m,n,k,pad", [(40, 64, 128, 8), (40, 64, 128, 6), (300, 256, 72, 16), (7, 9, 11, 3)])
def test_linear_strided_and_in_place(m, n, k, pad):
    rng = np.random.default_rng(m + pad)
    x, w = cols(rng, m, k, 2 * pad, "bf16"), tens(rng, (n, k), "bf16", std=k ** -0.5)
    y = cols(rng, m, n, 2 * pad, "bf16")
    whole = y._base.clone()
    yr, _ = ref.linear_fwd(host(x), host(w), None, host(y))
    out = ssd.linear_fwd(x, w, None, y, y=y)
    assert out is y and rel(host(y), yr) <= BAR["bf16"]
    assert torch.equal(y._base[:, :pad], whole[:, :pad]) and torch.equal(y._base[:, pad + n:], whole[:, pad + n:])


def test_linear_nonfinite_values_stay_in_their_rows():
    rng = np.random.default_rng(9)
    x, w = tens(rng, (200, 128), "bf16"), tens(rng, (192, 128), "bf16")
    x[3, 4] = float("nan")
    x[150, 7] = float("inf")
    y = ssd.linear_fwd(x, w, activation="relu")
    bad = ~torch.isfinite(y.float()).all(dim=1)
    assert bad[3] and torch.isnan(y[3].float()).all() and bad[150] and int(bad.sum()) == 2


@pytest.mark.parametrize("m,n,k", PRODUCT_SHAPES)
@pytest.mark.parametrize("d,act", [("bf16", "none"), ("bf16", "silu"), ("bf16", "gelu"), ("f32", "silu")])
def test_linear_bwd(m, n, k, d, act):
    rng = np.random.default_rng(m * 5 + n + k)
    x, w = tens(rng, (m, k), d), tens(rng, (n, k), d, std=k ** -0.5)
    dy = tens(rng, (m, n), d)
    p = tens(rng, (m, n), d) if act != "none" else None
    dx, dw, db = ssd.linear_bwd(dy, x, w, p, activation=act)
    dxr, dwr, dbr = ref.linear_bwd(host(dy), host(x), host(w), host(p) if p is not None else None, act)
    bar = BAR["f32"] if d == "f32" else (4e-3 if act == "none" else 8e-3)
    assert rel(host(dx), dxr) <= bar and rel(host(dw), dwr) <= bar
    dp = host(dy) * (ref.act_slope(host(p), act) if p is not None else 1.0)
    assert np.linalg.norm(host(db) - dbr) <= BAR["f32"] * np.linalg.norm(dp)
    again = ssd.linear_bwd(dy, x, w, p, activation=act)
    assert torch.equal(dx, again[0]) and torch.equal(dw, again[1]) and torch.equal(db, again[2])


def test_linear_bwd_parts_and_strides():
    rng = np.random.default_rng(11)
    m, n, k = 77, 40, 56
    x, w, dy = cols(rng, m, k, 8, "bf16"), tens(rng, (n, k), "bf16"), cols(rng, m, n, 24, "bf16")
    dxr, dwr, dbr = ref.linear_bwd(host(dy), host(x), host(w))
    dx, dw, db = ssd.linear_bwd(dy, x, w, need_dw=False, bias=False)
    assert dw is None and db is None and rel(host(dx), dxr) <= BAR["bf16"]
    dx, dw, db = ssd.linear_bwd(dy, x, w, need_dx=False)
    assert dx is None and rel(host(dw), dwr) <= BAR["bf16"] and rel(host(db), dbr) <= BAR["f32"]


def test_linear_no_tokens():
    x, w = torch.empty((0, 64), dtype=torch.bfloat16, device="cuda"), torch.ones((32, 64), dtype=torch.bfloat16, device="cuda")
    assert ssd.linear_fwd(x, w).shape == (0, 32)
    dx, dw, db = ssd.linear_bwd(torch.empty((0, 32), dtype=torch.bfloat16, device="cuda"), x, w)
    assert dx.shape == (0, 64) and torch.all(dw == 0) and torch.all(db == 0)
    y, _, rstd, _ = ssd.rmsnorm_fwd(x, torch.ones(64, device="cuda"))
    assert y.shape == (0, 64) and rstd.shape == (0,)


# ----------------------------------------------------------------- recurrence
def _scan_case(rng, cu, width, d, gate, parts_pad=0, mean=2.0, std=2.0):
    total = cu[-1]
    parts = 3 if gate else 2
    rows = tens(rng, (total, parts * width + parts_pad), d)
    rows[:, width:2 * width] = tens(rng, (total, width), d, std=std, mean=mean)
    x, g = rows[:, :width], rows[:, width:2 * width]
    z = rows[:, 2 * width:3 * width] if gate else None
    init = tens(rng, (len(cu) - 1, width))
    return x, g, z, init


def _check_scan(x, g, z, init, cu, d, packed, rng):
    n, width = len(cu) - 1, x.shape[1]
    hx, hg, hz = host(x), host(g), None if z is None else host(z)
    hi = host(init) if init is not None else np.zeros((n, width))
    yr, _, fr, before = ref.gated_fwd(hx, hg, hz, hi, cu)
    kw = {"cu_seqlens": cu} if packed else {}
    cut = (lambda t: t) if packed else (lambda t: None if t is None else t.unflatten(0, (n, -1)))
    y, f, kept = ssd.gated_scan_fwd(cut(x), cut(g), cut(z), init, return_checkpoints=True, **kw)
    assert y.dtype == DT[d] and f.dtype == torch.float32
    # states are one sum a channel: held against the size of their terms, which may cancel
    _, _, fsize, ksize = ref.gated_fwd(np.abs(hx), hg, None, np.abs(hi), cu)
    assert rel(host(y).reshape(yr.shape), yr) <= BAR[d]
    assert np.linalg.norm(host(f) - fr) <= BAR["f32"] * np.linalg.norm(fsize)
    assert np.linalg.norm(host(kept) - before[::64]) <= BAR["f32"] * np.linalg.norm(ksize[::64])
    y2, f2 = ssd.gated_scan_fwd(cut(x), cut(g), cut(z), init, **kw)
    # the order of the sums may follow the progress of other blocks: both results are held to the bar
    assert rel(host(y2).reshape(yr.shape), yr) <= BAR[d]
    assert np.linalg.norm(host(f2) - fr) <= BAR["f32"] * np.linalg.norm(fsize)
    dy, dfinal = tens(rng, x.shape, d), tens(rng, (n, width))
    dxr, dgr, dzr, dir_ = ref.gated_bwd(host(dy), hx, hg, hz, hi, host(dfinal), cu)
    dx, dg, dz, di = ssd.gated_scan_bwd(cut(dy), cut(x), cut(g), kept, cut(z), init, dfinal, **kw)
    assert rel(host(dx).reshape(dxr.shape), dxr) <= BAR[d]
    assert rel(host(dg).reshape(dgr.shape), dgr) <= BAR[d]
    # dinit is one sum a channel: held against the size of its terms, which may cancel
    dh = host(dy) if z is None else host(dy) * ref.silu(hz)
    size = ref.gated_bwd(np.abs(dh), hx, hg, None, hi, np.abs(host(dfinal)), cu)[3]
    assert np.linalg.norm(host(di) - dir_) <= BAR["f32"] * np.linalg.norm(size)
    if z is None:
        assert dz is None
    else:
        assert rel(host(dz).reshape(dzr.shape), dzr) <= BAR[d]
    ssd.last_device_error()


@pytest.mark.parametrize("n,length", [(1, 1), (5, 1), (3, 2), (2, 63), (1, 64), (2, 65), (1, 127), (1, 128), (3, 129),
                                      (2, 300), (1, 1000), (40, 7), (1, 5000)])
@pytest.mark.parametrize("width", [1, 2, 64, 65, 130])
@pytest.mark.parametrize("d,gate", [("f32", True), ("bf16", True), ("bf16", False)])
def test_recurrence(n, length, width, d, gate):
    rng = np.random.default_rng(n * 1000 + length + width)
    cu = [length * i for i in range(n + 1)]
    x, g, z, init = _scan_case(rng, cu, width, d, gate)
    _check_scan(x, g, z, init if n != 3 else None, cu, d, False, rng)


@pytest.mark.parametrize("lens", [[5], [0, 3, 0, 0, 64, 1, 0], [1] * 150, [63, 1, 64, 65, 200, 0], [700, 3, 1300],
                                  [64] * 9, [0, 0]])
@pytest.mark.parametrize("width,d,gate", [(8, "f32", False), (66, "bf16", True), (33, "bf16", False)])
def test_recurrence_packed(lens, width, d, gate):
    rng = np.random.default_rng(sum(lens) + width)
    cu = [0] + np.cumsum(lens).tolist()
    x, g, z, init = _scan_case(rng, cu, width, d, gate)
    _check_scan(x, g, z, init, cu, d, True, rng)


@pytest.mark.parametrize("mean,std", [(0.0, 60.0), (9.0, 0.5), (-9.0, 0.5)])
def test_recurrence_extreme_gates(mean, std):
    """Gates of 0 and 1 to fp32's precision, memories of one and of 8000 tokens."""
    rng = np.random.default_rng(int(mean) + 50)
    cu = [0, 1500]
    x, g, z, init = _scan_case(rng, cu, 40, "f32", True, mean=mean, std=std)
    _check_scan(x, g, z, init, cu, "f32", False, rng)


@pytest.mark.parametrize("pad", [1, 2, 8])
def test_recurrence_strided_gradients_into_one_matrix(pad):
    rng = np.random.default_rng(pad)
    cu, width = [0, 200], 48
    x, g, z, init = _scan_case(rng, cu, width, "bf16", True, parts_pad=pad)
    y, f, kept = ssd.gated_scan_fwd(x[None], g[None], z[None], init, return_checkpoints=True)
    dy = tens(rng, (1, 200, width), "bf16")
    grads = torch.full((1, 200, 3 * width + pad), 7.0, dtype=torch.bfloat16, device="cuda")
    dx, dg, dz, _ = ssd.gated_scan_bwd(dy, x[None], g[None], kept, z[None], init, None,
                                       dx=grads[..., :width], dg=grads[..., width:2 * width],
                                       dz=grads[..., 2 * width:3 * width])
    want = ref.gated_bwd(host(dy)[0], host(x), host(g), host(z), host(init), np.zeros((1, width)), cu)
    for got, w in zip((dx, dg, dz), want):
        assert rel(host(got)[0], w) <= BAR["bf16"]
    assert torch.all(grads[..., 3 * width:] == 7.0)


def test_recurrence_nan_stays_in_its_channel_and_sequence():
    rng = np.random.default_rng(3)
    cu = [0, 150, 400]
    x, g, z, init = _scan_case(rng, cu, 64, "f32", False)
    x[20, 5] = float("nan")
    y, f = ssd.gated_scan_fwd(x, g, None, init, cu_seqlens=cu)
    bad = torch.isnan(y)
    assert bad[20:150, 5].all() and int(bad.sum()) == 130 and int(torch.isnan(f).sum()) == 1


@pytest.mark.parametrize("rows,width,pad", [(1, 1, 0), (3, 66, 0), (256, 5120, 0), (7, 64, 8), (5, 33, 1)])
@pytest.mark.parametrize("d,gate", [("f32", True), ("bf16", True), ("bf16", False)])
def test_recurrence_step(rows, width, pad, d, gate):
    rng = np.random.default_rng(rows + width)
    x, g, z, _ = _scan_case(rng, [0, rows], width, d, gate, parts_pad=pad)
    state = tens(rng, (rows, width))
    cu = list(range(rows + 1))
    yr, hr, _, _ = ref.gated_fwd(host(x), host(g), None if z is None else host(z), host(state), cu)
    y = ssd.gated_state_update(state, x, g, z)
    assert rel(host(y), yr) <= BAR[d] and rel(host(state), hr) <= BAR["f32"]


def test_step_by_step_equals_the_scan():
    rng = np.random.default_rng(8)
    b, length, width = 3, 70, 96
    x, g, z, init = _scan_case(rng, [length * i for i in range(b + 1)], width, "f32", True)
    x, g, z = (t.unflatten(0, (b, length)) for t in (x, g, z))
    y, f = ssd.gated_scan_fwd(x, g, z, init)
    state = init.clone()
    for t in range(length):
        yt = ssd.gated_state_update(state, x[:, t], g[:, t], z[:, t])
        assert rel(host(yt), host(y[:, t])) <= BAR["f32"]
    assert rel(host(state), host(f)) <= BAR["f32"]


# --------------------------------------------------------- streams and refusals
def test_calls_follow_the_current_stream():
    """Inputs written on a side stream, calls on the same stream, no wait for the default one."""
    rng = np.random.default_rng(1)
    x, w = tens(rng, (64, 256), "bf16"), tens(rng, (256,))
    wl, g = tens(rng, (256, 256), "bf16"), tens(rng, (1, 64, 256), "bf16")
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        torch.cuda._sleep(20_000_000)
        x2 = x * 2
        y, _, _, _ = ssd.rmsnorm_fwd(x2, w)
        p = ssd.linear_fwd(y, wl)
        h, _ = ssd.gated_scan_fwd(p[None], g)
    s.synchronize()
    yr, _, _ = ref.norm_fwd(host(x) * 2, None, host(w), 1e-5)
    assert rel(host(y), yr) <= BAR["bf16"]
    assert rel(host(p), host(y) @ host(wl).T) <= BAR["bf16"]
    hr = ref.gated_fwd(host(p), host(g)[0], None, np.zeros((1, 256)), [0, 64])[0]
    assert rel(host(h)[0], hr) <= BAR["bf16"]


def test_calls_can_be_captured_in_a_graph():
    rng = np.random.default_rng(2)
    x, w = tens(rng, (1, 300, 128), "bf16"), tens(rng, (128,))
    wl = tens(rng, (384, 128), "bf16", std=0.1)

    def layer():
        y, _, _, _ = ssd.rmsnorm_fwd(x, w)
        p = ssd.linear_fwd(y, wl)
        return ssd.gated_scan_fwd(p[..., :128], p[..., 128:256], p[..., 256:])[0]
    want = layer().clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        layer()
    side.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer()
    for _ in range(3):
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert rel(host(out), host(want)) <= 1e-3     # the recurrence's sums may be joined in another order


def test_refusals():
    bf, f32 = torch.bfloat16, torch.float32
    x, w = torch.zeros((4, 64), dtype=bf, device="cuda"), torch.zeros((64,), device="cuda")
    wl = torch.zeros((32, 64), dtype=bf, device="cuda")
    with pytest.raises(ValueError):
        ssd.rmsnorm_fwd(x.cpu(), w)
    with pytest.raises(ValueError):
        ssd.rmsnorm_fwd(x, w[:32])
    with pytest.raises(TypeError):
        ssd.rmsnorm_fwd(x, w.to(bf))
    with pytest.raises(ValueError):
        ssd.rmsnorm_fwd(x.t(), torch.zeros((4,), device="cuda"))          # columns at a stride
    with pytest.raises(ssd.SsdError):
        ssd.rmsnorm_fwd(x, w, eps=-1.0)
    with pytest.raises(ssd.SsdError):
        ssd.rmsnorm_fwd(x.float(), w, x)                                   # a bf16 stream under f32 values
    with pytest.raises(ValueError):
        ssd.linear_fwd(x, wl[:, :32])
    with pytest.raises(ValueError):
        ssd.linear_fwd(x, wl, activation="tanh")
    with pytest.raises(ssd.SsdError):
        ssd.linear_fwd(x, wl, x_scale=torch.ones(4, device="cuda"))        # scales without 8-bit inputs
    x8, w8 = x.to(torch.float8_e4m3fn), wl.to(torch.float8_e4m3fn)
    with pytest.raises(ssd.SsdError):
        ssd.linear_fwd(x8, w8)                                             # 8-bit inputs without scales
    with pytest.raises(ssd.SsdError):
        ssd.linear_fwd(x.float(), wl.float(), out_dtype=bf)
    with pytest.raises(ssd.SsdError):
        ssd.linear_bwd(torch.zeros((4, 32), dtype=bf, device="cuda"), x, wl, activation="silu")   # no preact
    g = torch.zeros((1, 4, 64), dtype=bf, device="cuda")
    with pytest.raises(ValueError):
        ssd.gated_scan_fwd(x, x)
    with pytest.raises(ValueError):
        ssd.gated_scan_fwd(x, x, cu_seqlens=[0, 5])
    with pytest.raises(ssd.SsdError):
        ssd.gated_scan_fwd(x, x, cu_seqlens=[0, 3, 2, 4])
    with pytest.raises(TypeError):
        ssd.gated_scan_fwd(g, g.float())
    with pytest.raises(ValueError):
        ssd.gated_scan_bwd(g, g, g, None)
    with pytest.raises(ValueError):
        ssd.gated_scan_bwd(g, g, g, torch.zeros((2, 64), device="cuda"))
    with pytest.raises(TypeError):
        ssd.gated_state_update(torch.zeros((4, 64), dtype=bf, device="cuda"), x, x)
    with pytest.raises(ValueError):
        ssd.rmsnorm_fwd(torch.zeros((4, 64), device="cuda").as_strided((4, 64), (32, 1)), w.to(f32))   # rows overlap
