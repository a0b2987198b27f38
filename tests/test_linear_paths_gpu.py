"""The tensor-core product on each of its paths, with the whole epilogue (bias, scales,
activation, residual, values before the activation) and last rows and columns that are
not full, against the formulas in 64 bits.

Bars, derived before the first run: an output is rounded once to bf16, by at most 2^-8
of itself; the sums' 32 bits over k <= 5120 terms, and the residual's addition after
them, stay below 1e-4 of the terms' size, which is the outputs': 2^-8 + 1e-4 as
relative L2, and of the largest value for each value by itself (nothing is left out or
computed for another place).  An fp32 output has the latter part alone, 1e-4."""
import numpy as np
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import layer_ref as ref
from tests.gpu_util import host, rel

pytestmark = pytest.mark.gpu
FP8 = torch.float8_e4m3fn
BAR = {torch.bfloat16: 2.0 ** -8 + 1e-4, torch.float32: 1e-4}


def _values(rng, rows, cols, std=1.0):
    return torch.from_numpy(rng.standard_normal((rows, cols), dtype=np.float32) * np.float32(std)).cuda()


def _operand(rng, rows, k, dtype, std=1.0):
    t = _values(rng, rows, k, std)
    if dtype is not FP8:
        return t.to(dtype), None
    scale = t.abs().amax(dim=1) / 448.0
    return (t / scale[:, None]).to(FP8), scale


def _close(got, want, bar):
    wrong = np.abs(host(got) - want)
    assert np.linalg.norm(wrong) <= bar * np.linalg.norm(want)
    assert wrong.max() <= bar * np.abs(want).max()


def _check(m, n, k, dtype, out_dtype=torch.bfloat16, activation="silu"):
    rng = np.random.default_rng(m + 3 * n + k)
    x, xs = _operand(rng, m, k, dtype)
    w, ws = _operand(rng, n, k, dtype, k ** -0.5)
    bias, residual = _values(rng, 1, n)[0], _values(rng, m, n).to(out_dtype)
    y, p = ssd.linear_fwd(x, w, bias, residual, activation=activation, x_scale=xs, w_scale=ws,
                          out_dtype=out_dtype, return_preact=True)
    yr, pr = ref.linear_fwd(host(x), host(w), host(bias), host(residual), activation,
                            None if xs is None else host(xs), None if ws is None else host(ws))
    _close(y, yr, BAR[out_dtype])
    _close(p, pr, BAR[torch.bfloat16])
    bare = ssd.linear_fwd(x, w, x_scale=xs, w_scale=ws, out_dtype=out_dtype)
    _close(bare, pr - host(bias), BAR[out_dtype])
    ssd.last_device_error()


@pytest.mark.parametrize("dtype,k", [(torch.bfloat16, 2048), (FP8, 4096)])
@pytest.mark.parametrize("m,n", [
    (40, 200), (17, 8), (33, 1032),     # tokens as columns: features that end in a tile's first warp
    (200, 264), (130, 520), (100, 2560),   # one CTA's tiles: rows that end in the first warp, 8 columns in the last tile
    (1800, 1000),                       # pairs: the second CTA of the last row of tiles has no row
])
def test_sums_split_over_a_cluster(m, n, dtype, k):
    """Rows and columns past the end take no part in the exchange of sums."""
    _check(m, n, k, dtype)
    _check(m, n, k, dtype, torch.float32, "relu")


@pytest.mark.parametrize("wide", [4194240, 4194241, 4194303])
def test_most_columns_in_32_bits(wide):
    """Tiles of 64 columns past 65535: the last sizes below the limit of 2^22."""
    rng = np.random.default_rng(wide)
    x, w = _values(rng, 5, 3), _values(rng, wide, 3)
    y = ssd.linear_fwd(x, w)
    assert rel(host(y), host(x) @ host(w).T) <= 1e-5
    # the gradients of a product of as many inner values
    dy, x, w = _values(rng, 5, 2), _values(rng, 5, wide), _values(rng, 2, wide)
    dx, dw, _ = ssd.linear_bwd(dy, x, w, bias=False)
    assert rel(host(dx), host(dy) @ host(w)) <= 1e-5 and rel(host(dw), host(dy).T @ host(x)) <= 1e-5
    ssd.last_device_error()


# path, tokens, features, inner of a bf16 product; E4M3 has twice as many values in a block of k
FORWARD = [
    ("few", 16, 1003, 2048), ("few_split", 17, 200, 2048), ("few_split", 33, 1003, 2048), ("few_split", 64, 1000, 1000),
    ("split", 200, 264, 2048), ("split", 129, 1001, 1000), ("split_pairs", 1800, 1000, 2048),
    ("whole", 3000, 2100, 512), ("whole", 700, 2051, 264), ("pairs", 2200, 2000, 1000), ("whole", 2311, 1803, 1000), ("pairs", 2303, 2003, 1000),
    ("pairs_and_split", 2500, 2000, 4096), ("pairs_and_split", 2313, 2050, 4096),
]


@pytest.mark.parametrize("dtype,out_dtype,activation", [
    (torch.bfloat16, torch.bfloat16, "silu"), (torch.bfloat16, torch.float32, "relu"),
    (FP8, torch.bfloat16, "silu"), (FP8, torch.float32, "none")])
@pytest.mark.parametrize("path,m,n,k", FORWARD)
def test_forward_on_each_path(path, m, n, k, dtype, out_dtype, activation):
    k = 2 * k if dtype is FP8 else k
    assert ssd.linear_path(dtype, m, n, k) == path
    _check(m, n, k, dtype, out_dtype, activation)


# path, and a product of rows x columns by a sum over `terms`
ALONE = [("split", 200, 264, 2048), ("split_pairs", 1800, 1000, 2048), ("whole", 3000, 2104, 512),
         ("pairs", 2200, 2000, 1000), ("pairs_and_split", 2312, 2056, 4096)]


@pytest.mark.parametrize("path,rows,columns,terms", ALONE)
def test_dx_alone_on_each_path(path, rows, columns, terms):
    rng = np.random.default_rng(rows)
    assert ssd.linear_path(torch.bfloat16, rows, terms, columns, "dx") == path
    dy, w = _values(rng, rows, terms).bfloat16(), _values(rng, terms, columns, terms ** -0.5).bfloat16()
    x = torch.empty((rows, columns), dtype=torch.bfloat16, device="cuda")
    dx, dw, db = ssd.linear_bwd(dy, x, w, need_dw=False, bias=False)
    assert dw is None and db is None
    _close(dx, host(dy) @ host(w), BAR[torch.bfloat16])
    ssd.last_device_error()


@pytest.mark.parametrize("path,rows,columns,terms", ALONE)
@pytest.mark.parametrize("odd", [0, 3])
def test_dw_alone_on_each_path(path, rows, columns, terms, odd):
    rng = np.random.default_rng(rows + odd)
    tokens = terms - odd
    assert ssd.linear_path(torch.bfloat16, tokens, rows, columns, "dw") == path
    dy, x = _values(rng, tokens, rows).bfloat16(), _values(rng, tokens, columns).bfloat16()
    w = torch.empty((rows, columns), dtype=torch.bfloat16, device="cuda")
    dx, dw, _ = ssd.linear_bwd(dy, x, w, need_dx=False, bias=False)
    assert dx is None
    _close(dw, host(dy).T @ host(x), BAR[torch.bfloat16])
    ssd.last_device_error()


@pytest.mark.parametrize("path,tokens,features,inner", [
    ("together", 300, 1024, 1000), ("together", 2635, 2000, 1952), ("together", 700, 1003 // 8 * 8, 264),
    ("apart", 5000, 5000, 2600)])
@pytest.mark.parametrize("activation", ["none", "silu"])
def test_both_gradients_on_each_path(path, tokens, features, inner, activation):
    rng = np.random.default_rng(tokens)
    assert ssd.linear_path(torch.bfloat16, tokens, features, inner, "gradients") == path
    dy, x = _values(rng, tokens, features).bfloat16(), _values(rng, tokens, inner).bfloat16()
    w = _values(rng, features, inner, features ** -0.5).bfloat16()
    p = None if activation == "none" else _values(rng, tokens, features).bfloat16()
    dx, dw, db = ssd.linear_bwd(dy, x, w, p, activation=activation)
    want = ref.linear_bwd(host(dy), host(x), host(w), None if p is None else host(p), activation)
    bar = BAR[torch.bfloat16] if p is None else 2.0 ** -7 + 1e-4    # dp too is rounded once
    _close(dx, want[0], bar)
    _close(dw, want[1], bar)
    dp = host(dy) if p is None else host(dy) * ref.act_slope(host(p), activation)
    assert np.linalg.norm(host(db) - want[2]) <= 1e-5 * np.linalg.norm(dp)
    ssd.last_device_error()


def test_paths_of_other_types_and_sizes():
    assert ssd.linear_path(torch.float32, 100, 64, 64) == "fp32"
    assert ssd.linear_path(torch.float32, 4, 64, 64) == "fp32_few"
    assert ssd.linear_path(torch.bfloat16, 3, 64, 63) == "fp32_few"     # rows off 16 bytes
    assert ssd.linear_path(torch.bfloat16, 100, 64, 63) == "fp32"
    assert ssd.linear_path(torch.bfloat16, 100, 63, 64, "dx") == "fp32"
    assert ssd.linear_path(torch.bfloat16, 100, 63, 64, "gradients") == "apart"
    for bad in ((FP8, 64, 64, 64, "dx"), (torch.bfloat16, 0, 64, 64), (torch.bfloat16, 8, 64, 0)):
        with pytest.raises(ssd.SsdError):
            ssd.linear_path(*bad)
    with pytest.raises(ValueError):
        ssd.linear_path(torch.bfloat16, 8, 8, 8, "dy")
