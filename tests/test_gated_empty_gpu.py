"""A packed batch of very many empty sequences: their states are handed on, and nobody
waits for that."""
import numpy as np
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import layer_ref as ref
from tests.gpu_util import host, rel

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [2, 33])
def test_a_million_empty_sequences_hold_nobody_up(width):
    rng = np.random.default_rng(width)
    full, lens = {1: 70, 499_999: 3, 500_000: 200, 1_000_002: 65}, np.zeros(1_000_004, dtype=np.int64)
    for s, n in full.items():
        lens[s] = n
    cu = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    tokens, nseq = int(cu[-1]), lens.size
    new = lambda *shape: torch.from_numpy(rng.standard_normal(shape, dtype=np.float32)).cuda()   # noqa: E731
    x, g, dy, init, dfinal = new(tokens, width), new(tokens, width), new(tokens, width), new(nseq, width), new(nseq, width)
    offsets = {"cu_seqlens": cu, "cu_seqlens_dev": torch.from_numpy(cu).cuda()}
    ssd.last_device_error()
    # a wait lasts some microseconds; 2 ms are far above that and far below a pass over all sequences
    ssd.debug_inject_fault(ssd.FAULT_NONE, 2_000_000)
    try:
        y, final, kept = ssd.gated_scan_fwd(x, g, None, init, return_checkpoints=True, **offsets)
        dx, _, _, dinit = ssd.gated_scan_bwd(dy, x, g, kept, None, init, dfinal, **offsets)
        ssd.last_device_error()                       # no wait ran out
    finally:
        ssd.debug_inject_fault(ssd.FAULT_NONE, 0)
    some = sorted(full)
    ends = np.concatenate([[0], np.cumsum(lens[some])]).tolist()
    hi, hd = host(init)[some], host(dfinal)[some]
    yr, _, fr, _ = ref.gated_fwd(host(x), host(g), None, hi, ends)
    dxr, _, _, dir_ = ref.gated_bwd(host(dy), host(x), host(g), None, hi, hd, ends)
    assert rel(host(y), yr) <= 1e-5 and rel(host(final)[some], fr) <= 1e-5
    assert rel(host(dx), dxr) <= 1e-5 and rel(host(dinit)[some], dir_) <= 1e-5
    empty = torch.from_numpy(lens == 0).cuda()
    assert torch.equal(final[empty], init[empty]) and torch.equal(dinit[empty], dfinal[empty])
    assert ssd.gated_scan_fwd(x, g, **offsets)[1][empty].abs().max() == 0
