"""The linear layer's kernels keep their values in registers: the compiler's resource remarks show no scratch memory, which
spilled registers would take. Needs hipcc, no GPU."""
import os
import re
import subprocess

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


@pytest.mark.parametrize("source", ["pipe_norm.hip", "pipe_gemm_fp8.hip", "pipe_gemm_w4.hip"])
def test_no_scratch_memory(source, tmp_path):
    found = remarks(source, os.path.join(tmp_path, "out.s"))
    assert {k: v for k, v in found.items() if v} == {}
