"""The most dynamic shared memory that a kernel may be launched with is an attribute of the
kernel, shared by all host threads: a launch sets it to what the kernel's largest call takes,
never to the call's own size, which another thread's call of the same kernel may exceed between
setting and launch.  Checked on the sources: the value is a constant of the kernel."""
import glob
import os
import re

import pytest

from tests.test_early_launch_host import CSRC, _code

CONSTANT = re.compile(r"(\(int\)\s*)?(k[A-Z]\w*|\w+::kBytes|join_bytes\(r\)|(scan|seg)_smem<\w+>\(\)|simt_smem_bytes\(kMostStates\))")


def _values(code):
    """The last arguments of the calls that set the attribute."""
    for m in re.finditer(r"cudaFuncAttributeMaxDynamicSharedMemorySize,", code):
        depth, end = 1, m.end()
        while depth:
            depth += {"(": 1, ")": -1}.get(code[end], 0)
            end += 1
        yield re.sub(r"[\s\\]+", " ", code[m.end():end - 1]).strip()


@pytest.mark.parametrize("name", sorted(os.path.basename(f) for f in glob.glob(os.path.join(CSRC, "*.cu"))))
def test_the_attribute_is_the_kernel_s(name):
    for value in _values(_code(name)):
        assert CONSTANT.fullmatch(value), value
