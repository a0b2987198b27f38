"""The recurrence's bounded waits, made to run out without any GPU fault: the
host-set test hook lets the walk's first tile publish nothing, so the tiles
behind it give up at a short limit.  The host reads SSD_ERR_TIMEOUT, and the
next call on the same context is correct."""
import numpy as np
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import layer_ref as ref
from tests.gpu_util import host, rel

pytestmark = pytest.mark.gpu

TIMEOUT = 4   # SSD_ERR_TIMEOUT


@pytest.mark.parametrize("backward", [False, True])
def test_withheld_run_times_out_then_next_call_is_correct(backward):
    gen = torch.Generator(device="cuda").manual_seed(3)
    x, g, dy = (torch.empty((1, 700, 96), device="cuda").normal_(generator=gen) for _ in range(3))
    _, _, kept = ssd.gated_scan_fwd(x, g, return_checkpoints=True)
    call = (lambda: ssd.gated_scan_bwd(dy, x, g, kept)[0]) if backward else (lambda: ssd.gated_scan_fwd(x, g)[0])
    ssd.last_device_error()                           # start from a clear error word
    ssd.debug_inject_fault(ssd.FAULT_WITHHOLD_SIGNAL, 2_000_000)   # 2 ms limit
    try:
        call()                                        # outputs undefined
        torch.cuda.synchronize()
    finally:
        ssd.debug_inject_fault(ssd.FAULT_NONE, 0)
    with pytest.raises(ssd.SsdError) as err:
        ssd.last_device_error()
    assert err.value.code == TIMEOUT
    ssd.last_device_error()                           # read once, then clear
    zero = np.zeros((1, 96))
    want = (ref.gated_bwd(host(dy)[0], host(x)[0], host(g)[0], None, zero, zero, [0, 700])[0] if backward
            else ref.gated_fwd(host(x)[0], host(g)[0], None, zero, [0, 700])[0])
    assert rel(host(call())[0], want) <= 1e-5
    ssd.last_device_error()
