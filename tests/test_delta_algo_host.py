"""Host-side checks of the delta rule's choice of kernels in the C ABI (no GPU needed)."""
import pytest

from tests.test_layer_abi_host import BAD, BF16, F32, FP8, INVALID, P, UNSUPPORTED, WORKSPACE, lib  # noqa: F401

AUTO, SIMT, TC = 0, 1, 2
SIZES = (1000, 3, 4, 64, 128, 2)        # tokens, nseq, heads, headdim, dstate, groups


def _fwd(lib, algo, **kw):  # noqa: F811
    a = dict(q=P[0], k=P[1], v=P[2], g=P[3], beta=P[4], d=BF16, nseq=2, length=100, cu=None, cud=None, heads=4, p=64,
             n=128, groups=2, qs=256, ks=256, vs=256, scale=0.1, init=None, o=P[5], os=256, final=P[6], kept=P[7],
             ws=P[8], wb=1 << 40)
    a.update(kw)
    return lib.ssd_delta_scan_fwd_algo(algo, *a.values(), None)


def _bwd(lib, algo, **kw):  # noqa: F811
    a = dict(do=P[0], q=P[1], k=P[2], v=P[3], g=P[4], beta=P[5], d=BF16, nseq=2, length=100, cu=None, cud=None, heads=4,
             p=64, n=128, groups=2, dos=256, qs=256, ks=256, vs=256, scale=0.1, kept=P[6], dfinal=None, dq=P[7],
             dqs=256, dk=P[8], dks=256, dv=P[9], dvs=256, dg=P[10], db=P[11], dinit=None, ws=P[12], wb=1 << 40)
    a.update(kw)
    return lib.ssd_delta_scan_bwd_algo(algo, *a.values(), None)


@pytest.mark.parametrize("algo", [-1, 3])
def test_unknown_choices(lib, algo):  # noqa: F811
    assert _fwd(lib, algo) == INVALID == _bwd(lib, algo)
    assert lib.ssd_delta_scan_workspace_bytes_algo(algo, BF16, *SIZES) == BAD
    assert lib.ssd_delta_scan_bwd_workspace_bytes_algo(algo, BF16, *SIZES) == BAD


@pytest.mark.parametrize("kw", [dict(d=F32), dict(n=100, qs=200, ks=200), dict(p=60), dict(n=136, groups=1),
                                dict(q=P[0] + 2), dict(vs=260)])
def test_what_the_tensor_cores_do_not_take(lib, kw):  # noqa: F811
    assert _fwd(lib, TC, **kw) == UNSUPPORTED == _bwd(lib, TC, **kw)


def test_other_checks_come_with_every_choice(lib):  # noqa: F811
    for algo in (AUTO, SIMT, TC):
        assert _fwd(lib, algo, q=None) == INVALID == _bwd(lib, algo, do=None)
        assert _fwd(lib, algo, d=FP8) == UNSUPPORTED == _bwd(lib, algo, d=FP8)
        assert _bwd(lib, algo, length=0) == 0
    assert _bwd(lib, SIMT, ws=None) == WORKSPACE == _bwd(lib, SIMT, wb=1000)


def test_workspaces(lib):  # noqa: F811
    fwd, bwd = lib.ssd_delta_scan_workspace_bytes_algo, lib.ssd_delta_scan_bwd_workspace_bytes_algo
    for d in (BF16, F32):
        assert fwd(AUTO, d, *SIZES) == lib.ssd_delta_scan_workspace_bytes(d, *SIZES)
        assert bwd(AUTO, d, *SIZES) == lib.ssd_delta_scan_bwd_workspace_bytes(d, *SIZES)
        assert fwd(SIMT, d, *SIZES) == 0 < bwd(SIMT, d, *SIZES)
        assert bwd(AUTO, d, *SIZES) == max(bwd(SIMT, d, *SIZES), bwd(TC, d, *SIZES))
    assert fwd(TC, BF16, *SIZES) == fwd(AUTO, BF16, *SIZES) > 0 and bwd(TC, BF16, *SIZES) > 0
    for odd in ((1000, 3, 4, 60, 128, 2), (1000, 3, 4, 64, 136, 2), (0, 3, 4, 64, 128, 2)):
        assert fwd(TC, BF16, *odd) == 0 == bwd(TC, BF16, *odd)
    for query in (fwd, bwd):
        assert query(TC, BF16, 1000, 3, 5, 64, 128, 2) == BAD
