"""8-bit products whose scales are far from 1: the sum is scaled by the one and then by
the other, so their product, which may be below or above fp32's range, is never taken."""
import numpy as np
import pytest
import torch

import state_space_model_chunked_gb300 as ssd
from tests import layer_ref as ref
from tests.gpu_util import host, rel

pytestmark = pytest.mark.gpu


# one token, few, tokens as columns, split, whole, unaligned rows; 1e-5: fp32 sums and two roundings
@pytest.mark.parametrize("m,n,k", [(1, 64, 512), (16, 40, 512), (40, 200, 4096), (200, 264, 4096), (3000, 2100, 1024),
                                   (2, 40, 333), (70, 40, 333)])
@pytest.mark.parametrize("sx,sw", [(1e-22, 1e-22), (1e-30, 3e-12), (1e20, 1e10)])
def test_scales_far_from_one(m, n, k, sx, sw):
    rng = np.random.default_rng(m)
    x, w = (torch.from_numpy(np.clip(rng.standard_normal((r, k), dtype=np.float32) * 100, -448, 448)).cuda().to(torch.float8_e4m3fn)
            for r in (m, n))
    xs = torch.from_numpy((rng.uniform(1, 2, m) * sx).astype(np.float32)).cuda()
    ws = torch.from_numpy((rng.uniform(1, 2, n) * sw).astype(np.float32)).cuda()
    if sx > 1:                                         # 0 times an infinite product of scales would be NaN
        ws[1::2] *= 1e9
        keep = w.float()
        keep[1::2] = 0.0
        w = keep.to(torch.float8_e4m3fn)
    y = ssd.linear_fwd(x, w, x_scale=xs, w_scale=ws, out_dtype=torch.float32)
    want, _ = ref.linear_fwd(host(x), host(w), x_scale=xs.double().cpu().numpy(), w_scale=ws.double().cpu().numpy())
    top = np.abs(want).max()
    assert rel(host(y) / top, want / top) <= 1e-5
