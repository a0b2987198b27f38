"""Host-side checks of the layer's operators in the C ABI (no GPU needed): bad
arguments come back before anything is enqueued, and the workspace queries
answer for valid sizes and refuse others."""
import ctypes

import numpy as np
import pytest

import state_space_model_chunked_gb300 as ssd
from state_space_model_chunked_gb300 import build as ssd_build

OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 5
F32, BF16, FP8 = 0, 1, 2
BAD = ctypes.c_size_t(-1).value
P = [0x10000 * (i + 1) for i in range(16)]       # fake, aligned device addresses


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.load()


def _norm_fwd(lib, **kw):
    a = dict(x=P[0], r=P[1], w=P[2], eps=1e-5, xd=BF16, sd=BF16, od=BF16, rows=4, width=64, xs=64, rs=64, y=P[3],
             ro=P[4], rstd=P[5], scale=None)
    a.update(kw)
    return lib.ssd_rmsnorm_fwd(a["x"], a["r"], a["w"], a["eps"], a["xd"], a["sd"], a["od"], a["rows"], a["width"],
                               a["xs"], a["rs"], a["y"], a["ro"], a["rstd"], a["scale"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(rstd=None), INVALID),
    (dict(ro=None), INVALID), (dict(od=FP8), INVALID),            # 8 bits without scales
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(rows=-1), INVALID), (dict(width=0), INVALID),
    (dict(xs=63), INVALID), (dict(rs=10), INVALID), (dict(x=P[0] + 1), INVALID), (dict(xd=9), INVALID),
    (dict(xd=FP8), UNSUPPORTED), (dict(xd=F32), UNSUPPORTED),     # a bf16 stream under f32 values
    (dict(rows=1 << 31), UNSUPPORTED), (dict(width=1 << 24, xs=1 << 24, rs=1 << 24), UNSUPPORTED),
    (dict(rows=0), OK),
])
def test_norm_fwd_checks(lib, kw, expect):
    assert _norm_fwd(lib, **kw) == expect


def _norm_bwd(lib, **kw):
    a = dict(dy=P[0], s=P[1], w=P[2], rstd=P[3], dr=P[4], d=BF16, sd=F32, rows=4, width=64, ys=64, ss=64, drs=64,
             dx=P[5], ds=P[6], dw=P[7], ws=P[8], wb=1 << 30)
    a.update(kw)
    return lib.ssd_rmsnorm_bwd(a["dy"], a["s"], a["w"], a["rstd"], a["dr"], a["d"], a["sd"], a["rows"], a["width"],
                               a["ys"], a["ss"], a["drs"], a["dx"], a["ds"], a["dw"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dy=None), INVALID), (dict(dw=None), INVALID), (dict(dx=None), INVALID), (dict(ss=32), INVALID),
    (dict(drs=32), INVALID), (dict(d=FP8), UNSUPPORTED), (dict(d=F32, sd=BF16), UNSUPPORTED),
])
def test_norm_bwd_checks(lib, kw, expect):
    assert _norm_bwd(lib, **kw) == expect


def _linear_fwd(lib, **kw):
    a = dict(x=P[0], xsc=None, w=P[1], wsc=None, b=P[2], r=P[3], act=1, d=BF16, od=BF16, m=8, n=64, k=32, xs=32, rs=64,
             y=P[4], ys=64, pre=None)
    a.update(kw)
    return lib.ssd_linear_fwd(a["x"], a["xsc"], a["w"], a["wsc"], a["b"], a["r"], a["act"], a["d"], a["od"], a["m"],
                              a["n"], a["k"], a["xs"], a["rs"], a["y"], a["ys"], a["pre"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(act=4), INVALID),
    (dict(act=-1), INVALID), (dict(m=-1), INVALID), (dict(n=0), INVALID), (dict(k=0), INVALID), (dict(xs=31), INVALID),
    (dict(ys=63), INVALID), (dict(rs=63), INVALID), (dict(xsc=P[5], wsc=P[6]), INVALID),
    (dict(d=FP8), INVALID),                                        # 8 bits without scales
    (dict(d=FP8, xsc=P[5]), INVALID), (dict(d=FP8, xsc=P[5], wsc=P[6], x=P[0] + 2), INVALID),
    (dict(od=FP8), UNSUPPORTED), (dict(d=F32), UNSUPPORTED), (dict(n=1 << 22, ys=1 << 22, rs=1 << 22), UNSUPPORTED),
    (dict(m=1 << 31), UNSUPPORTED), (dict(m=0), OK),
])
def test_linear_fwd_checks(lib, kw, expect):
    assert _linear_fwd(lib, **kw) == expect


def _linear_bwd(lib, **kw):
    a = dict(dy=P[0], x=P[1], w=P[2], pre=P[3], act=1, d=BF16, m=8, n=64, k=32, ys=64, xs=32, dx=P[4], dw=P[5], db=P[6],
             ws=P[7], wb=1 << 30)
    a.update(kw)
    return lib.ssd_linear_bwd(a["dy"], a["x"], a["w"], a["pre"], a["act"], a["d"], a["m"], a["n"], a["k"], a["ys"],
                              a["xs"], a["dx"], a["dw"], a["db"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dy=None), INVALID), (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(pre=None), INVALID),
    (dict(act=0), INVALID),                                        # values before no activation
    (dict(ys=63), INVALID), (dict(xs=31), INVALID), (dict(d=FP8), UNSUPPORTED), (dict(k=1 << 22, xs=1 << 22), UNSUPPORTED),
])
def test_linear_bwd_checks(lib, kw, expect):
    assert _linear_bwd(lib, **kw) == expect


def _cu(offsets):
    a = np.ascontiguousarray(offsets, dtype=np.int32)
    return a, a.ctypes.data_as(ctypes.c_void_p)


def _scan_fwd(lib, **kw):
    a = dict(x=P[0], g=P[1], z=P[2], d=BF16, n=2, L=20, cu=None, cud=None, width=64, xs=64, gs=64, zs=64, init=P[3],
             y=P[4], ys=64, fin=P[5], ck=None, ws=None, wb=0)
    a.update(kw)
    return lib.ssd_gated_scan_fwd(a["x"], a["g"], a["z"], a["d"], a["n"], a["L"], a["cu"], a["cud"], a["width"], a["xs"],
                                  a["gs"], a["zs"], a["init"], a["y"], a["ys"], a["fin"], a["ck"], a["ws"], a["wb"], None)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), INVALID), (dict(g=None), INVALID), (dict(y=None), INVALID), (dict(n=0), INVALID), (dict(L=-1), INVALID),
    (dict(width=0), INVALID), (dict(xs=60), INVALID), (dict(gs=60), INVALID), (dict(zs=60), INVALID), (dict(ys=60), INVALID),
    (dict(init=P[3] + 2), INVALID), (dict(cud=P[6]), INVALID), (dict(d=FP8), UNSUPPORTED),
    (dict(n=1 << 16, L=1 << 16), UNSUPPORTED), (dict(width=1 << 21, xs=1 << 21, gs=1 << 21, zs=1 << 21, ys=1 << 21), UNSUPPORTED),
    (dict(L=2000), WORKSPACE),
])
def test_gated_scan_checks(lib, kw, expect):
    assert _scan_fwd(lib, **kw) == expect


@pytest.mark.parametrize("offsets", [[1, 5, 9], [0, 5, 3]])
def test_gated_scan_refuses_bad_offsets(lib, offsets):
    keep, cu = _cu(offsets)
    assert _scan_fwd(lib, cu=cu, cud=P[6]) == INVALID
    assert _scan_fwd(lib, cu=cu, cud=None) == INVALID


def test_gated_bwd_checks(lib):
    def call(dy=P[0], ck=P[4], dz=P[7], dzs=64, dxs=64, wb=0, L=20):
        return lib.ssd_gated_scan_bwd(dy, P[1], P[2], P[3], BF16, 2, L, None, None, 64, 64, 64, 64, 64, None, ck, None,
                                      P[5], dxs, P[6], 64, dz, dzs, None, None, wb, None)
    assert call(dy=None) == INVALID
    assert call(ck=None) == INVALID
    assert call(dz=None) == INVALID
    assert call(dzs=3) == INVALID
    assert call(dxs=3) == INVALID
    assert call(L=2000) == WORKSPACE


def test_state_update_checks(lib):
    def call(state=P[0], x=P[1], d=BF16, rows=3, width=64, xs=64, y=P[3]):
        return lib.ssd_gated_state_update(state, x, P[2], None, d, rows, width, xs, 64, 64, y, None)
    assert call(state=None) == INVALID and call(x=None) == INVALID and call(y=None) == INVALID
    assert call(rows=-1) == INVALID and call(width=0) == INVALID and call(xs=10) == INVALID
    assert call(d=FP8) == UNSUPPORTED and call(d=7) == INVALID
    assert call(rows=0) == OK


def test_workspace_queries(lib):
    assert lib.ssd_rmsnorm_bwd_workspace_bytes(-1, 64) == BAD
    assert lib.ssd_rmsnorm_bwd_workspace_bytes(10, 0) == BAD
    assert lib.ssd_linear_bwd_workspace_bytes(FP8, 0, 8, 8, 8) == BAD
    assert lib.ssd_linear_bwd_workspace_bytes(BF16, 9, 8, 8, 8) == BAD
    assert lib.ssd_linear_bwd_workspace_bytes(BF16, 1, 0, 8, 8) == 0
    # the rounded dp of an activation, then the partial column sums
    none, silu = (lib.ssd_linear_bwd_workspace_bytes(BF16, act, 1000, 96, 64) for act in (0, 1))
    assert silu - none == (1000 * 96 * 2 + 255) // 256 * 256
    assert lib.ssd_gated_scan_workspace_bytes(BF16, 64, 100) == 0          # one tile: nothing to join
    assert lib.ssd_gated_scan_workspace_bytes(BF16, -1, 100) == BAD
    assert lib.ssd_gated_scan_workspace_bytes(FP8, 10, 100) == BAD
    # a ticket, and a word of 8 bytes for every tile of 64 tokens and channel
    assert lib.ssd_gated_scan_workspace_bytes(F32, 640, 100) == (256 + 10 * 100 * 8 + 255) // 256 * 256
