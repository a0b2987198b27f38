"""The gradients of the delta rule take the workspace of the kernels that run, not of those that
other addresses would take."""
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests.test_delta_algo_gpu import shifted
from tests.test_delta_gpu import inputs

pytestmark = pytest.mark.gpu

TOKENS, NSEQ, GROUPS, HEADS, P, N = 2000, 2, 2, 4, 128, 128
SIZES = (TOKENS, NSEQ, HEADS, P, N, GROUPS)


def setup(dtype):
    x, init, do, dfinal = inputs(5, TOKENS, NSEQ, GROUPS, HEADS, P, N, dtype)
    b = {name: t.unflatten(0, (NSEQ, -1)) for name, t in x.items()}
    kept = ssd.delta_scan_fwd(*b.values(), init, return_checkpoints=True)[2]
    return b, do.unflatten(0, (NSEQ, -1)), kept, dfinal


def made_by(call):
    """The bytes of the arrays that a call makes, less its outputs."""
    count = lambda: torch.cuda.memory_stats()["allocated_bytes.all.allocated"]   # noqa: E731
    before = count()
    out = call()
    return count() - before - sum(t.numel() * t.element_size() for t in out)


@pytest.mark.parametrize("long_way", [False, True])
def test_memory_of_a_call(long_way):
    b, do, kept, dfinal = setup("bf16")
    tc, simt = (ssd.delta_scan_bwd_workspace_bytes(torch.bfloat16, *SIZES, algo=a) for a in (ssd.ALGO_TCGEN05, ssd.ALGO_SIMT))
    assert tc != simt and ssd.delta_scan_bwd_workspace_bytes(torch.bfloat16, *SIZES) == max(tc, simt)
    out = dict(dg=torch.empty_like(b["g"])) if long_way else {}
    given = sum(t.numel() * t.element_size() for t in out.values())
    slack = 1 << 20         # (the allocator's rounding)
    for args, need in ((b, tc), (dict(b, k=shifted(b["k"])), simt)):
        got = made_by(lambda: ssd.delta_scan_bwd(do, *args.values(), kept, dfinal, **out)) + given
        assert need - slack <= got <= need + slack, (got, need)
    full, do, kept, dfinal = setup("f32")
    need = ssd.delta_scan_bwd_workspace_bytes(torch.float32, *SIZES)
    assert abs(made_by(lambda: ssd.delta_scan_bwd(do, *full.values(), kept, dfinal, **out)) + given - need) <= slack


@pytest.mark.parametrize("algo", [ssd.ALGO_AUTO, ssd.ALGO_SIMT, ssd.ALGO_TCGEN05])
def test_a_workspace_of_that_size_is_enough(algo):
    b, do, kept, dfinal = setup("bf16")
    need = ssd.delta_scan_bwd_workspace_bytes(torch.bfloat16, *SIZES, algo=algo or ssd.ALGO_TCGEN05)
    buf = torch.full((need + 4096,), 0x5a, dtype=torch.uint8, device="cuda")
    want = ssd.delta_scan_bwd(do, *b.values(), kept, dfinal, algo=algo)
    got = ssd.delta_scan_bwd(do, *b.values(), kept, dfinal, algo=algo, workspace=buf[:need])
    assert all(torch.equal(g, w) for g, w in zip(got, want))
    assert torch.all(buf[need:] == 0x5a)
