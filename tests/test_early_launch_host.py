"""Kernels that may start while the one in front of them in the stream still runs read
its results after griddepcontrol.wait, with ordinary loads: a read-only-cache load
(`__ldg`, ld.global.nc) is defined only for memory that nothing writes during the
kernel's lifetime, and that begins before the wait.  Checked on the sources of the
operators that are launched so."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "state_space_model_chunked_gb300", "csrc")


def _code(name):
    text = open(os.path.join(CSRC, name)).read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", ["linear_few.cu", "linear_tc.cu", "linear_simt.cu", "rmsnorm.cu", "act.cuh", "vec.cuh"])
def test_no_read_only_cache_loads_behind_an_early_launch(name):
    code = _code(name)
    assert not re.search(r"__ldg\s*\(|ld\.global\.nc|const\s+\w+\s*\*\s*__restrict__", code)
