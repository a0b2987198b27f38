"""The bounded wait of the layer norm's row-a-warp kernel, made to run out without any GPU
fault: the host-set test hook keeps the first row's copy from being complete.  Its warp gives
up at the limit and ends, the other rows are as they should be, the host reads
SSD_ERR_TIMEOUT, and the next call on the same context is correct."""
import pytest
import torch

import state_space_model_chunked_gb300 as ssd

pytestmark = pytest.mark.gpu

TIMEOUT = 4   # SSD_ERR_TIMEOUT


@pytest.mark.parametrize("residual", [False, True])
def test_withheld_copy_times_out_then_next_call_is_correct(residual):
    rows, width = 20000, 256        # several rows a warp
    x = torch.randn((rows, width), device="cuda").bfloat16()
    w, r = torch.randn(width, device="cuda"), torch.randn((rows, width), device="cuda").bfloat16() if residual else None
    call = lambda: ssd.layernorm_fwd(x, w, None, r, out_dtype=torch.float8_e4m3fn)   # noqa: E731
    want = call()
    ssd.last_device_error()                           # start from a clear error word
    mean, rstd, scale = (torch.full((rows,), float("nan"), device="cuda") for _ in range(3))
    ssd.debug_inject_fault(ssd.FAULT_WITHHOLD_SIGNAL, 2_000_000)   # 2 ms limit
    try:
        got = ssd.layernorm_fwd(x, w, None, r, out_dtype=torch.float8_e4m3fn, mean=mean, rstd=rstd, scale=scale)
        torch.cuda.synchronize()
    finally:
        ssd.debug_inject_fault(ssd.FAULT_NONE, 0)
    with pytest.raises(ssd.SsdError) as err:
        ssd.last_device_error()
    assert err.value.code == TIMEOUT
    ssd.last_device_error()                           # read once, then clear
    same = [(a.view(torch.uint8) == b.view(torch.uint8)).view(rows, -1).all(1) for a, b in zip((got[0], got[2], got[3], got[4]), (want[0], want[2], want[3], want[4]))]
    # the first row is not written, nor are those that its warp would have gone on with
    lost = ~torch.stack(same).all(0)
    assert 1 <= int(lost.sum()) <= 40 and lost[0]
    again = call()
    assert torch.equal(again[0].view(torch.uint8), want[0].view(torch.uint8)) and torch.equal(again[4], want[4])
    ssd.last_device_error()
