"""8-bit rows of the norm so small that their scale is not an fp32 number: zeros, not NaN."""
import pytest
import torch

import state_space_model_chunked_gb300 as ssd

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("width", [64, 2560, 8191, 33000])      # vectors, scalars, the two-pass form
def test_rows_below_any_scale_are_zero(width):
    x = torch.zeros((3, width), device="cuda")
    x[0, 1::2] = 1.0                    # y = sqrt(2) 2^-145: its scale would be 7e-47
    x[2] = -2.0                         # y = -2^-145
    w = torch.full((width,), 2.0 ** -145, device="cuda")
    y, _, _, scale = ssd.rmsnorm_fwd(x, w, out_dtype=torch.float8_e4m3fn)
    assert (y.float() == 0).all() and (scale == 1).all()
    y, _, _, scale = ssd.rmsnorm_fwd(x, w * 2.0 ** 10, out_dtype=torch.float8_e4m3fn)
    v = y.float() * scale[:, None]      # sqrt(2) 2^-135 = 3.2e-41 and -2^-135, scales of some 2^-144
    assert (v[0, 0::2] == 0).all() and (v[0, 1::2] > 3e-41).all() and (v[2] < -2e-41).all() and (v[1] == 0).all()
