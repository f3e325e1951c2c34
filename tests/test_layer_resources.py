"""Layer norm's and the microscaled 4-bit form's kernels keep their values in registers, as the linear layer's others do. Needs
hipcc, no GPU."""
import os
from concurrent.futures import ThreadPoolExecutor

import pytest

from tests.test_linear_resources import remarks

SOURCES = ["pipe_layernorm.hip", "pipe_mx_quant.hip", "pipe_gemm_mx.hip"]


@pytest.fixture(scope="module")
def found(tmp_path_factory):
    where = tmp_path_factory.mktemp("remarks")
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        return dict(zip(SOURCES, ex.map(lambda s: remarks(s, os.path.join(where, s + ".s")), SOURCES)))


@pytest.mark.parametrize("source", SOURCES)
def test_no_scratch_memory(source, found):
    assert {k: v for k, v in found[source].items() if v} == {}
