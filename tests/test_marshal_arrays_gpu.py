"""Arrays that compiled marshalling makes: torch's dispatch modes see them, and fill them where
deterministic algorithms ask for that."""
import pytest
import torch
from torch.utils._python_dispatch import TorchDispatchMode

import state_space_model_chunked_gb300 as ssd

pytestmark = pytest.mark.gpu


class Made(TorchDispatchMode):
    """The bytes of the arrays made under it."""

    def __init__(self):
        super().__init__()
        self.bytes = []

    def __torch_dispatch__(self, func, types, args=(), kwargs=None):
        out = func(*args, **(kwargs or {}))
        if func is torch.ops.aten.empty.memory_format:
            self.bytes.append(out.numel() * out.element_size())
        return out


def calls():
    bf = dict(device="cuda", dtype=torch.bfloat16)
    x, w, table = torch.randn((16, 64), **bf), torch.ones(64, device="cuda"), torch.randn((50, 64), **bf)
    t = torch.arange(16, device="cuda")
    wide = torch.randn((32, 64), **bf)
    q, g = torch.randn((1, 70, 2, 64), **bf), -torch.rand((1, 70, 2), device="cuda")
    state = torch.zeros((1, 2, 64, 64), device="cuda")
    y, _, mean, rstd, _ = ssd.layernorm_fwd(x, w)
    rms = ssd.rmsnorm_fwd(x, w)[2]
    kept = ssd.delta_scan_fwd(q, q, q, g, g, return_checkpoints=True)[2]
    return {"rmsnorm_fwd": lambda: ssd.rmsnorm_fwd(x, w), "rmsnorm_bwd": lambda: ssd.rmsnorm_bwd(x, x, w, rms),
            "linear_fwd": lambda: ssd.linear_fwd(x, wide), "linear_bwd": lambda: ssd.linear_bwd(torch.ones((16, 32), **bf), x, wide),
            "gated_scan_fwd": lambda: ssd.gated_scan_fwd(q[..., 0, :].contiguous(), q[..., 1, :].contiguous()),
            "layernorm_fwd": lambda: ssd.layernorm_fwd(x, w), "layernorm_bwd": lambda: ssd.layernorm_bwd(x, x, w, mean, rstd),
            "embedding_fwd": lambda: ssd.embedding_fwd(t, table), "embedding_bwd": lambda: ssd.embedding_bwd(x, t, 50),
            "delta_scan_fwd": lambda: ssd.delta_scan_fwd(q, q, q, g, g, return_checkpoints=True),
            "delta_scan_bwd": lambda: ssd.delta_scan_bwd(q, q, q, q, g, g, kept),
            "delta_state_update": lambda: ssd.delta_state_update(state, q[:, 0], q[:, 0], q[:, 0], g[:, 0], g[:, 0])}


def outputs(out):
    return [t for t in (out if isinstance(out, tuple) else (out,)) if t is not None]


@pytest.mark.parametrize("name", ["rmsnorm_fwd", "rmsnorm_bwd", "linear_fwd", "linear_bwd", "gated_scan_fwd", "layernorm_fwd",
                                  "layernorm_bwd", "embedding_fwd", "embedding_bwd", "delta_scan_fwd", "delta_scan_bwd",
                                  "delta_state_update"])
def test_a_dispatch_mode_sees_what_is_made(name):
    call = calls()[name]
    with Made() as made:
        out = call()
    want = {t.data_ptr(): t.numel() * t.element_size() for t in outputs(out)}      # (one array may be two outputs)
    for size in want.values():
        assert size in made.bytes
        made.bytes.remove(size)


def test_places_that_nothing_writes_are_filled_where_torch_is_asked_to():
    q, g = torch.randn((130, 2, 64), device="cuda", dtype=torch.bfloat16), -torch.rand((130, 2), device="cuda")
    cu = [0, 65, 65, 130]       # of 130 // 64 + 3 places, two sequences' two each are written
    torch.use_deterministic_algorithms(True)
    try:
        kept = ssd.delta_scan_fwd(q, q, q, g, g, cu_seqlens=cu, return_checkpoints=True)[2]
    finally:
        torch.use_deterministic_algorithms(False)
    assert kept.shape[0] == 5 and torch.isnan(kept).flatten(1).all(1).sum() == 1 and torch.isfinite(kept).flatten(1).all(1).sum() == 4
