"""As in test_early_launch_host.py, for the layer norm, the embedding and the delta rule's
single token: no read-only-cache loads in kernels that may start before the one in front of
them has ended."""
import re

import pytest

from tests.test_early_launch_host import _code


@pytest.mark.parametrize("name", ["layernorm.cu", "norm_rows.cuh", "embedding.cu", "delta_step.cu"])
def test_no_read_only_cache_loads(name):
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|const\s+\w+\s*\*\s*__restrict__", _code(name))
