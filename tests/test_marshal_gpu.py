"""The compiled marshalling hands on the errors of its arguments as they are."""
import pytest
import torch

import state_space_model_chunked_gb300 as ssd

pytestmark = pytest.mark.gpu


def test_a_flag_without_a_truth_value():
    x = torch.zeros((1, 70, 64), device="cuda")
    with pytest.raises(RuntimeError, match="Boolean value"):
        ssd.gated_scan_fwd(x, x, return_checkpoints=torch.ones(2))
    w, dy = torch.zeros((8, 64), device="cuda"), torch.zeros((70, 8), device="cuda")
    with pytest.raises(RuntimeError, match="Boolean value"):
        ssd.linear_bwd(dy, x[0], w, bias=torch.ones(2))
