"""The layer norm of rows enough for a warp each (8-bit output, 16 rows an SM and more), in the
ways of test_layernorm_gpu.py that need many rows here: column ranges of wider matrices whose rows
start on 16 bytes, every pair of types, rows of NaN, infinities, one constant and tiny values, the
residual in place; and more than 2^31 values.  Bars as there."""
import numpy as np
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import model_ref as ref
from tests.gpu_util import host, rel
from tests.test_layernorm_gpu import BAR, DT, cols, tens

pytestmark = pytest.mark.gpu


def check(x, w, b, r, got):
    y, s, mean, rstd, scale = got
    yr, sr, mr, rr = ref.layernorm_fwd(host(x), None if r is None else host(r), host(w), None if b is None else host(b), 1e-5)
    assert np.linalg.norm(host(mean) - mr) <= BAR["f32"] * np.linalg.norm(np.sqrt((sr * sr).mean(axis=-1)))
    assert rel(host(rstd), rr) <= BAR["f32"]
    if s is not None:
        assert rel(host(s), sr) <= (4e-3 if s.dtype == torch.bfloat16 else 1e-5)
    top, sc = np.abs(yr).max(axis=-1), host(scale)[:, None]
    assert rel(host(scale), top / 448.0) <= BAR["f32"]
    assert np.all(np.abs(host(y) * sc - yr) <= np.abs(yr) * 2.0 ** -4 + 1e-5 * top[:, None] + sc * 2.0 ** -10)


def on_16(t):
    return t.data_ptr() % 16 == 0 and t.stride(0) * t.element_size() % 16 == 0


@pytest.mark.parametrize("rows,width", [(2432, 8), (2432, 264), (2433, 512), (3000, 1024), (2440, 1544), (5003, 2048),
                                        (2600, 2560), (2450, 4096), (2450, 2816)])
@pytest.mark.parametrize("xd,rd,pad", [("bf16", None, 0), ("bf16", "bf16", 0), ("bf16", "bf16", 16), ("bf16", "f32", 0), ("bf16", "f32", 16),
                                       ("f32", None, 0), ("f32", None, 8), ("f32", "f32", 0), ("f32", "f32", 8)])
@pytest.mark.parametrize("bias", [True, False])
def test_types_and_strides(rows, width, xd, rd, pad, bias):
    rng = np.random.default_rng(rows + width + pad)
    x, w = cols(rng, rows, width, pad, xd, mean=0.5), tens(rng, (width,), std=0.3, mean=1.0)
    b, r = tens(rng, (width,), std=0.5) if bias else None, cols(rng, rows, width, pad, rd, std=3.0) if rd else None
    assert on_16(x) and (r is None or on_16(r)) and x.is_contiguous() == (pad == 0)
    check(x, w, b, r, ssd.layernorm_fwd(x, w, b, r, eps=1e-5, out_dtype=DT["fp8"]))


@pytest.mark.parametrize("width", [264, 1544, 2560])
@pytest.mark.parametrize("xd,rd", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
def test_the_residual_in_place(width, xd, rd):
    rng = np.random.default_rng(width)
    x, w, r = tens(rng, (2500, width), xd), tens(rng, (width,)), tens(rng, (2500, width), rd, std=3.0)
    want = ssd.layernorm_fwd(x, w, None, r, out_dtype=DT["fp8"])
    got = ssd.layernorm_fwd(x, w, None, r, out_dtype=DT["fp8"], residual_out=r)
    assert got[1] is r
    for a, c in zip(got, want):
        assert torch.equal(a.view(torch.uint8), c.view(torch.uint8))


@pytest.mark.parametrize("width", [264, 2560])
@pytest.mark.parametrize("xd", ["bf16", "f32"])
def test_rows_of_all_kinds_stay_to_themselves(width, xd):
    rng = np.random.default_rng(width + 1)
    x, w, b = tens(rng, (6000, width), xd), tens(rng, (width,), std=0.3, mean=1.0), tens(rng, (width,))
    x[1] = 4.0
    x[2, 17], x[2500, width - 1] = float("nan"), float("nan")
    x[3, 5], x[4000, 0] = float("inf"), float("-inf")
    lost = torch.zeros(6000, dtype=torch.bool, device="cuda")
    lost[[2, 3, 2500, 4000]] = True
    y, _, mean, rstd, scale = ssd.layernorm_fwd(x, w, b, out_dtype=DT["fp8"])
    assert torch.isnan(y[lost].float()).all() and torch.isnan(scale[lost]).all() and torch.isnan(rstd[lost]).all()
    kept = ~lost
    kept[1] = False         # (a constant row's rstd is eps's alone)
    check(x[kept], w, b, None, (y[kept], None, mean[kept], rstd[kept], scale[kept]))
    # a constant row is its bias
    assert abs(scale[1].item() * 448 - b.abs().max().item()) <= 1e-5 * b.abs().max().item()


@pytest.mark.parametrize("weight", [1e-31, 1e-38, 1e-44])
def test_outputs_below_the_scales_range(weight):
    """Weights that make rows whose scale has no reciprocal in fp32, or is none."""
    rng = np.random.default_rng(3)
    x, w = tens(rng, (2500, 512), "f32"), torch.full((512,), weight, device="cuda")
    y, _, _, _, scale = ssd.layernorm_fwd(x, w, out_dtype=DT["fp8"])
    few = ssd.layernorm_fwd(x[:100], w, out_dtype=DT["fp8"])       # a CTA each
    yr = ref.layernorm_fwd(host(x), None, host(w), None, 1e-5)[0]
    top = np.abs(yr).max(axis=-1)
    step = 2.0 ** -149                                             # fp32's last subnormal
    assert torch.isfinite(y.float()).all() and torch.isfinite(scale).all()
    got = host(y) * host(scale)[:, None]
    # an E4M3 step of the value, the scale's own rounding on 448 of it, and two fp32 roundings
    assert np.all(np.abs(got - yr) <= np.abs(yr) * 2.0 ** -4 + 448 * step + (top / 448 + step)[:, None] * 2.0 ** -10 + 1e-5 * top[:, None])
    assert torch.equal(few[4] == 1.0, scale[:100] == 1.0)


def test_values_beyond_32_bits():
    """Rows past the 2^31st value, each against the same by itself, forward and backward."""
    rows, width = 840000, 2560
    assert rows * width > 2 ** 31
    x = torch.randn((rows, width), device="cuda", dtype=torch.bfloat16)
    w, b = torch.randn(width, device="cuda"), torch.randn(width, device="cuda")
    tail = slice(rows - 3000, rows)
    for out in (DT["fp8"], DT["bf16"]):
        y, s, mean, rstd, scale = ssd.layernorm_fwd(x, w, b, x, out_dtype=out)
        part = ssd.layernorm_fwd(x[tail].clone(), w, b, x[tail].clone(), out_dtype=out)
        for whole, few in zip((y, s, mean, rstd, scale), part):
            assert whole is few or torch.equal(whole[tail].view(torch.uint8), few.view(torch.uint8))
        del y, part
    dx, ds, dw, db = ssd.layernorm_bwd(x, s, w, mean, rstd, x)
    few = ssd.layernorm_bwd(x[tail].clone(), s[tail].clone(), w, mean[tail].clone(), rstd[tail].clone(), x[tail].clone())
    assert torch.equal(dx[tail], few[0]) and ds is dx
    half = rows // 2
    parts = [ssd.layernorm_bwd(x[i], s[i], w, mean[i], rstd[i], x[i])[2:] for i in (slice(0, half), slice(half, rows))]
    for whole, one, two in zip((dw, db), *parts):
        assert rel(host(whole), host(one) + host(two)) <= 1e-5
