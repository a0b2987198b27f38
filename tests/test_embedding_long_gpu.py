"""The embedding with more than 2^31 values on either side, against parts of it."""
import pytest
import torch

import state_space_model_chunked_gb300 as ssd

pytestmark = pytest.mark.gpu


def test_values_beyond_32_bits():
    vocab, width, count = 1100000, 2048, 1060000
    assert vocab * width > 2 ** 31 and count * width > 2 ** 31
    table = torch.randn((vocab, width), device="cuda", dtype=torch.bfloat16)
    t = torch.randint(vocab, (count,), device="cuda", generator=torch.Generator(device="cuda").manual_seed(1))
    t[-1], t[-2], t[0] = vocab - 1, -1, vocab - 2
    y = ssd.embedding_fwd(t, table)
    assert torch.all(y[-2] == 0)
    real = t >= 0
    for part in (slice(0, 2000), slice(count - 2000, count)):
        rows = t[part]
        assert torch.equal(y[part][real[part]], table[rows[real[part]]])
    # the gradient of rows of ones counts a row's tokens (up to 256 of them exactly, in bf16)
    y.fill_(1.0)
    dtable = ssd.embedding_bwd(y, t, vocab)
    counts = torch.bincount(t[real], minlength=vocab)
    assert int(counts.max()) <= 256
    for part in (slice(0, 3000), slice(vocab - 3000, vocab)):
        assert torch.equal(dtable[part], counts[part, None].to(torch.bfloat16).expand(-1, width))
    assert torch.equal(dtable[:, -1], counts.to(torch.bfloat16))
