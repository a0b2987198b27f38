"""The tensor-core delta rule's bounded waits, made to run out without any GPU fault: the
host-set test hook keeps the first product of the first CTA from being announced.  Its
warps give up at the limit, let its copies and products in flight complete and end; the
host reads SSD_ERR_TIMEOUT, and the next call on the same context is correct."""
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import model_ref as ref
from tests.gpu_util import host, rel
from tests.test_delta_gpu import BAR, STATE, batched, inputs

pytestmark = pytest.mark.gpu

TIMEOUT = 4   # SSD_ERR_TIMEOUT


@pytest.mark.parametrize("backward", [False, True])
@pytest.mark.parametrize("limit_ns", [1, 3_000, 20_000, 2_000_000])
@pytest.mark.parametrize("length,p,n", [(300, 128, 128), (40, 64, 64), (1700, 64, 64)])      # the last one in parts
def test_withheld_product_times_out_then_next_call_is_correct(length, p, n, limit_ns, backward):
    x, init, do, dfinal = inputs(length, length, 1, 1, 3, p, n, "bf16")
    b = batched(x, 1)
    o, final, kept = ssd.delta_scan_fwd(*b.values(), init, return_checkpoints=True)
    ssd.last_device_error()                           # start from a clear error word
    ssd.debug_inject_fault(ssd.FAULT_WITHHOLD_SIGNAL, limit_ns)
    try:
        if backward:                                  # outputs undefined
            ssd.delta_scan_bwd(do[None], *b.values(), kept, dfinal)
        else:
            ssd.delta_scan_fwd(*b.values(), init)
        torch.cuda.synchronize()
    finally:
        ssd.debug_inject_fault(ssd.FAULT_NONE, 0)
    with pytest.raises(ssd.SsdError) as err:
        ssd.last_device_error()
    assert err.value.code == TIMEOUT
    ssd.last_device_error()                           # read once, then clear
    if backward:
        got = ssd.delta_scan_bwd(do[None], *b.values(), kept, dfinal)
        grads = ref.delta_bwd(host(do), *map(host, x.values()), host(init), host(dfinal), [0, length], n ** -0.5)
        assert all(rel(host(g).reshape(w.shape), w) <= max(BAR["bf16"], STATE["bf16"]) for g, w in zip(got, grads))
    else:
        o, final = ssd.delta_scan_fwd(*b.values(), init)
    want, last, _ = ref.delta_fwd(*map(host, x.values()), host(init), [0, length], n ** -0.5)
    assert rel(host(o)[0], want) <= BAR["bf16"] and rel(host(final), last) <= STATE["bf16"]
    ssd.last_device_error()
