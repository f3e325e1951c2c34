"""The linear layer's kernels keep their values in registers: the compiler's resource remarks show no scratch memory, which
spilled registers would take. Needs hipcc, no GPU."""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from async_stage_tile_amd import build


def remarks(source, out):
    """Scratch bytes a lane of each kernel of a source file."""
    cmd = build.compile_command(source, out, [])
    cmd.remove("-fPIC")
    cmd[cmd.index("-c")] = "-S"
    res = subprocess.run([*cmd, "--offload-device-only", "-Rpass-analysis=kernel-resource-usage"], capture_output=True,
                         text=True)
    assert res.returncode == 0, res.stderr[-2000:]
    names = re.findall(r"Function Name: (\S+)", res.stderr)
    scratch = [int(v) for v in re.findall(r"ScratchSize \[bytes/lane\]: (\d+)", res.stderr)]
    assert len(names) == len(scratch) > 0
    return dict(zip(names, scratch))


SOURCES = ["pipe_norm.hip", "pipe_gemm_fp8.hip", "pipe_gemm_w4.hip"]


@pytest.fixture(scope="module")
def found(tmp_path_factory):
    where = tmp_path_factory.mktemp("remarks")
    with ThreadPoolExecutor(len(SOURCES)) as ex:
        return dict(zip(SOURCES, ex.map(lambda s: remarks(s, os.path.join(where, s + ".s")), SOURCES)))


@pytest.mark.parametrize("source", SOURCES)
def test_no_scratch_memory(source, found):
    assert {k: v for k, v in found[source].items() if v} == {}
