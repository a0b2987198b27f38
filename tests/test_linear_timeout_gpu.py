"""The tensor-core product's bounded waits, made to run out without any GPU fault: the
host-set test hook keeps the first accumulator from being announced.  Its CTA gives up
at the limit, lets its copies and products in flight complete (also where the limit is
shorter than a copy takes) and ends; the host reads SSD_ERR_TIMEOUT, and the next call
on the same context is correct."""
import numpy as np
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests.gpu_util import host, rel

pytestmark = pytest.mark.gpu

TIMEOUT = 4   # SSD_ERR_TIMEOUT


def _values(rng, rows, cols):
    return torch.from_numpy(rng.standard_normal((rows, cols), dtype=np.float32)).cuda().bfloat16()


@pytest.mark.parametrize("limit_ns", [1, 20_000, 2_000_000])
@pytest.mark.parametrize("m,n,k,backward", [
    (40, 200, 4096, False),             # few tokens, k split over a cluster
    (200, 264, 4096, False),            # one CTA's tiles, k split
    (3000, 2100, 512, False),           # one CTA's tiles, whole
    (1800, 1000, 2048, False),          # pairs, k split
    (9000, 2560, 2048, False),          # pairs, whole, many tiles each
    (2635, 1000, 1952, True),           # both gradients
])
def test_withheld_accumulator_times_out_then_next_call_is_correct(m, n, k, backward, limit_ns):
    rng = np.random.default_rng(m + n)
    x, w = _values(rng, m, k), _values(rng, n, k)
    dy = _values(rng, m, n) if backward else None
    call = (lambda: ssd.linear_bwd(dy, x, w, bias=False)[0]) if backward else (lambda: ssd.linear_fwd(x, w))
    ssd.last_device_error()                           # start from a clear error word
    ssd.debug_inject_fault(ssd.FAULT_WITHHOLD_SIGNAL, limit_ns)
    try:
        call()                                        # outputs undefined
        torch.cuda.synchronize()
    finally:
        ssd.debug_inject_fault(ssd.FAULT_NONE, 0)
    with pytest.raises(ssd.SsdError) as err:
        ssd.last_device_error()
    assert err.value.code == TIMEOUT
    ssd.last_device_error()                           # read once, then clear
    want = host(dy) @ host(w) if backward else host(x) @ host(w).T
    assert rel(host(call()), want) <= 4e-3            # rounded once to bf16
    ssd.last_device_error()
