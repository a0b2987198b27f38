"""Rows of one bf16 value: their sums are exact in fp32, so the mean is that value, what is left
of it is zero, and with it y without a bias."""
import pytest
import torch

import state_space_model_chunked_gb300 as ssd

pytestmark = pytest.mark.gpu

VALUES = [4.0, 0.1, -3.3, 7.96875, 1.9921875, 250.0, 1e-3, -1e4]


@pytest.mark.parametrize("out", [torch.float8_e4m3fn, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("x_dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("width", [7, 96, 264, 520, 776, 1544, 2047, 2560, 2816, 4096, 8184, 33000])
@pytest.mark.parametrize("rows", [8, 2432])
def test_their_mean_is_the_value(rows, width, x_dtype, out):
    values = torch.tensor(VALUES, device="cuda").bfloat16()
    x = values.repeat(rows // 8)[:, None].expand(-1, width).to(x_dtype).contiguous()
    y, _, mean, rstd, scale = ssd.layernorm_fwd(x, torch.randn(width, device="cuda"), out_dtype=out)
    assert torch.equal(mean, x[:, 0].float())
    assert torch.all(y.float() == 0) and (scale is None or torch.all(scale == 1.0))
    assert torch.allclose(rstd, torch.full_like(rstd, 1e-5 ** -0.5), rtol=1e-6)
