"""Host-side checks of the layer norm, the embedding and the delta rule in the C ABI (no GPU
needed): bad arguments come back before anything is enqueued, and the workspace queries answer
for sizes that are handled and refuse others."""
import numpy as np
import pytest

from tests.test_layer_abi_host import (BAD, BF16, F32, FP8, INVALID, OK, P, UNSUPPORTED, WORKSPACE,  # noqa: F401
                                       lib)

I32, I64 = 0, 1


def _layernorm_fwd(lib, **kw):  # noqa: F811
    a = dict(x=P[0], r=P[1], w=P[2], b=P[3], eps=1e-5, xd=BF16, sd=BF16, od=BF16, rows=4, width=64, xs=64, rs=64,
             y=P[4], ro=P[5], mean=P[6], rstd=P[7], scale=None)
    a.update(kw)
    return lib.ssd_layernorm_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(x=None), INVALID), (dict(w=None), INVALID), (dict(y=None), INVALID), (dict(mean=None), INVALID),
    (dict(rstd=None), INVALID), (dict(ro=None), INVALID), (dict(od=FP8), INVALID),      # 8 bits without scales
    (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID), (dict(rows=-1), INVALID), (dict(width=0), INVALID),
    (dict(xs=63), INVALID), (dict(rs=10), INVALID), (dict(x=P[0] + 1), INVALID), (dict(b=P[3] + 2), INVALID),
    (dict(mean=P[6] + 1), INVALID), (dict(xd=9), INVALID), (dict(od=-1), INVALID),
    (dict(xd=FP8), UNSUPPORTED), (dict(xd=F32), UNSUPPORTED),       # a bf16 stream under f32 values
    (dict(rows=1 << 31), UNSUPPORTED), (dict(width=1 << 24, xs=1 << 24, rs=1 << 24), UNSUPPORTED),
    (dict(rows=0), OK), (dict(rows=0, x=None, y=None), OK),
])
def test_layernorm_fwd_checks(lib, kw, expect):  # noqa: F811
    assert _layernorm_fwd(lib, **kw) == expect


def _layernorm_bwd(lib, **kw):  # noqa: F811
    a = dict(dy=P[0], s=P[1], w=P[2], mean=P[3], rstd=P[4], dr=P[5], d=BF16, sd=F32, rows=4, width=64, ys=64, ss=64,
             drs=64, dx=P[6], ds=P[7], dw=P[8], db=P[9], ws=P[10], wb=1 << 30)
    a.update(kw)
    return lib.ssd_layernorm_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dy=None), INVALID), (dict(mean=None), INVALID), (dict(dw=None), INVALID), (dict(dx=None), INVALID),
    (dict(db=P[9] + 1), INVALID), (dict(ss=32), INVALID), (dict(drs=32), INVALID), (dict(d=FP8), UNSUPPORTED),
    (dict(d=F32, sd=BF16), UNSUPPORTED), (dict(rows=1 << 31), UNSUPPORTED),
])
def test_layernorm_bwd_checks(lib, kw, expect):  # noqa: F811
    assert _layernorm_bwd(lib, **kw) == expect


def _embedding_fwd(lib, **kw):  # noqa: F811
    a = dict(t=P[0], it=I64, table=P[1], td=BF16, od=F32, count=5, vocab=100, width=24, scale=1.0, y=P[2])
    a.update(kw)
    return lib.ssd_embedding_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(t=None), INVALID), (dict(table=None), INVALID), (dict(y=None), INVALID), (dict(it=2), INVALID),
    (dict(t=P[0] + 4), INVALID), (dict(table=P[1] + 1), INVALID), (dict(count=-1), INVALID), (dict(vocab=0), INVALID),
    (dict(width=0), INVALID), (dict(scale=float("inf")), INVALID), (dict(td=FP8), UNSUPPORTED),
    (dict(od=FP8), UNSUPPORTED), (dict(count=(1 << 31) - 2048), UNSUPPORTED), (dict(vocab=1 << 30), UNSUPPORTED),
    (dict(width=1 << 24), UNSUPPORTED), (dict(count=0), OK), (dict(count=0, t=None, y=None), OK),
])
def test_embedding_fwd_checks(lib, kw, expect):  # noqa: F811
    assert _embedding_fwd(lib, **kw) == expect


def _embedding_bwd(lib, **kw):  # noqa: F811
    a = dict(dy=P[0], t=P[1], it=I32, d=BF16, od=F32, count=5, vocab=100, width=24, ys=24, scale=1.0, dt=P[2], ws=P[3],
             wb=1 << 40)
    a.update(kw)
    return lib.ssd_embedding_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(dy=None), INVALID), (dict(t=None), INVALID), (dict(dt=None), INVALID), (dict(ys=23), INVALID),
    (dict(dy=P[0] + 1), INVALID), (dict(t=P[1] + 2), INVALID), (dict(ws=None), WORKSPACE), (dict(wb=8), WORKSPACE),
    (dict(ws=P[3] + 16), INVALID), (dict(d=FP8), UNSUPPORTED), (dict(od=FP8), UNSUPPORTED), (dict(scale=float("nan")), INVALID),
])
def test_embedding_bwd_checks(lib, kw, expect):  # noqa: F811
    assert _embedding_bwd(lib, **kw) == expect


def _delta_fwd(lib, **kw):  # noqa: F811
    a = dict(q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], d=BF16, nseq=2, length=100, cu=None, cud=None, heads=4, p=64,
             n=128, groups=2, qs=256, ks=256, vs=256, scale=0.1, init=None, o=P[5], os=256, final=P[6], kept=P[7],
             ws=P[8], wb=1 << 40)
    a.update(kw)
    return lib.ssd_delta_scan_fwd(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(q=None), INVALID), (dict(k=None), INVALID), (dict(v=None), INVALID), (dict(g=None), INVALID),
    (dict(beta=None), INVALID), (dict(o=None), INVALID), (dict(q=P[0] + 1), INVALID), (dict(g=P[3] + 2), INVALID),
    (dict(init=P[9] + 2), INVALID), (dict(final=P[6] + 1), INVALID), (dict(kept=P[7] + 3), INVALID),
    (dict(heads=3), INVALID),                   # no whole number of heads a group
    (dict(heads=0), INVALID), (dict(groups=0), INVALID), (dict(p=0), INVALID), (dict(n=0), INVALID),
    (dict(nseq=0), INVALID), (dict(length=-1), INVALID), (dict(qs=255), INVALID), (dict(ks=1), INVALID),
    (dict(vs=255), INVALID), (dict(os=255), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(ws=None), WORKSPACE), (dict(wb=1000), WORKSPACE), (dict(ws=P[8] + 16), INVALID), (dict(d=9), INVALID),
    (dict(d=FP8), UNSUPPORTED), (dict(n=257, qs=600, ks=600), UNSUPPORTED), (dict(p=(1 << 14) + 1), UNSUPPORTED),
    (dict(nseq=1 << 16, length=1 << 15), UNSUPPORTED),
])
def test_delta_fwd_checks(lib, kw, expect):  # noqa: F811
    assert _delta_fwd(lib, **kw) == expect


@pytest.mark.parametrize("cu", [[0, 60, 50, 100], [1, 60, 100], [0, -5, 100]])
def test_delta_offsets(lib, cu):  # noqa: F811
    host = np.array(cu, dtype=np.int32)
    kw = dict(nseq=len(cu) - 1, length=0, cu=host.ctypes.data, cud=P[9])
    assert _delta_fwd(lib, **kw) == INVALID
    assert _delta_fwd(lib, **dict(kw, cud=None)) == INVALID


def _delta_bwd(lib, **kw):  # noqa: F811
    a = dict(do=P[0], q=P[1], k=P[2], v=P[3], g=P[4], beta=P[5], d=F32, nseq=2, length=100, cu=None, cud=None, heads=4,
             p=64, n=128, groups=2, dos=256, qs=256, ks=256, vs=256, scale=0.1, kept=P[6], dfinal=None, dq=P[7],
             dqs=256, dk=P[8], dks=256, dv=P[9], dvs=256, dg=P[10], db=P[11], dinit=None, ws=P[12], wb=1 << 40)
    a.update(kw)
    return lib.ssd_delta_scan_bwd(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(do=None), INVALID), (dict(kept=None), INVALID), (dict(dq=None), INVALID), (dict(dk=None), INVALID),
    (dict(dv=None), INVALID), (dict(dg=None), INVALID), (dict(db=None), INVALID), (dict(dos=10), INVALID),
    (dict(dqs=255), INVALID), (dict(dks=255), INVALID), (dict(dvs=255), INVALID), (dict(dinit=P[13] + 1), INVALID),
    (dict(dfinal=P[13] + 2), INVALID), (dict(do=P[0] + 2), INVALID), (dict(ws=None), WORKSPACE),
    (dict(wb=1000), WORKSPACE), (dict(d=FP8), UNSUPPORTED), (dict(length=0), OK),
])
def test_delta_bwd_checks(lib, kw, expect):  # noqa: F811
    assert _delta_bwd(lib, **kw) == expect


def _delta_step(lib, **kw):  # noqa: F811
    a = dict(s=P[0], sd=F32, so=P[0], q=P[1], k=P[2], v=P[3], g=P[4], beta=P[5], d=BF16, batch=3, heads=4, p=64, n=128,
             groups=2, qs=256, ks=256, vs=256, scale=0.1, o=P[6])
    a.update(kw)
    return lib.ssd_delta_state_update(*a.values(), None)


@pytest.mark.parametrize("kw,expect", [
    (dict(s=None), INVALID), (dict(so=None), INVALID), (dict(q=None), INVALID), (dict(o=None), INVALID),
    (dict(s=P[0] + 2), INVALID), (dict(batch=-1), INVALID), (dict(heads=5), INVALID), (dict(qs=200), INVALID),
    (dict(vs=200), INVALID), (dict(scale=float("inf")), INVALID), (dict(sd=7), INVALID),
    (dict(sd=FP8), UNSUPPORTED), (dict(sd=BF16, d=F32), UNSUPPORTED), (dict(n=300, qs=900, ks=900), UNSUPPORTED),
    (dict(batch=0), OK), (dict(batch=0, s=None, q=None), OK),
])
def test_delta_step_checks(lib, kw, expect):  # noqa: F811
    assert _delta_step(lib, **kw) == expect


def test_workspace_queries(lib):  # noqa: F811
    assert lib.ssd_layernorm_bwd_workspace_bytes(-1, 64) == BAD == lib.ssd_layernorm_bwd_workspace_bytes(4, 0)
    assert lib.ssd_embedding_bwd_workspace_bytes(0, 10, 8) == 0
    assert lib.ssd_embedding_bwd_workspace_bytes(7, 10, 8) not in (0, BAD)
    assert lib.ssd_embedding_bwd_workspace_bytes(7, 0, 8) == BAD == lib.ssd_embedding_bwd_workspace_bytes(-1, 10, 8)
    fwd, bwd = lib.ssd_delta_scan_workspace_bytes, lib.ssd_delta_scan_bwd_workspace_bytes
    sizes = (1000, 3, 4, 64, 128, 2)
    assert fwd(F32, *sizes) == 0 and fwd(BF16, *sizes) not in (0, BAD)
    assert bwd(F32, *sizes) not in (0, BAD) and bwd(BF16, *sizes) not in (0, BAD)
    for query in (fwd, bwd):
        assert query(BF16, 0, 3, 4, 64, 128, 2) == 0        # no tokens, no work
        for bad in ((1000, 0, 4, 64, 128, 2), (-1, 3, 4, 64, 128, 2), (1000, 3, 5, 64, 128, 2),
                    (1000, 3, 4, 64, 257, 2), (1000, 3, 4, 0, 128, 2), (1 << 31, 3, 4, 64, 128, 2)):
            assert query(BF16, *bad) == BAD
