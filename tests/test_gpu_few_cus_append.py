"""The tests of test_gpu_paged_append.py on one compute unit, so that small calls take the instances
that the host otherwise chooses for many rows or units."""
import pytest

import moe_grouped_gemm_fp32_amd as fg
from test_gpu_paged_append import *  # noqa: F401,F403  (its tests, its marker)
from test_gpu_paged_append import pytestmark  # noqa: F401


@pytest.fixture(autouse=True)
def one_cu():
    fg.set_num_cus(1)
    yield
    fg.set_num_cus(0)
