"""The query of a product's path refuses what the product refuses, without a GPU."""
import pytest

import state_space_model_chunked_gb300 as ssd
from state_space_model_chunked_gb300 import build as ssd_build

F32, BF16, FP8 = 0, 1, 2


@pytest.fixture(scope="module")
def lib():
    ssd_build.build()
    return ssd.load()


@pytest.mark.parametrize("args", [
    (4, BF16, 8, 8, 8), (-1, BF16, 8, 8, 8), (0, 3, 8, 8, 8), (0, BF16, 0, 8, 8), (0, BF16, -1, 8, 8), (0, BF16, 8, 0, 8),
    (0, BF16, 8, 8, 0), (0, BF16, 8, 1 << 22, 8), (0, BF16, (1 << 31) - 256, 8, 8), (1, FP8, 8, 8, 8),
    (3, BF16, 8, 8, 1 << 22)])
def test_path_query_refuses(lib, args):
    assert lib.ssd_linear_path(*args) == -1


def test_names_follow_the_header():
    import os
    import re
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "ssd.h")).read()
    from state_space_model_chunked_gb300.layer_ops import PATHS, PRODUCTS
    paths = dict(re.findall(r"SSD_PATH_([A-Z0-9_]+) = (\d+)", text))
    assert [p.upper() for p in PATHS] == sorted(paths, key=lambda p: int(paths[p]))
    products = {k.lower(): int(v) for k, v in re.findall(r"SSD_PRODUCT_([A-Z]+) = (\d+)", text)}
    assert products == PRODUCTS
