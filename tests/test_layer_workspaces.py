"""Workspaces of the microscaled 4-bit product that hold no partial products: the largest products lay both operands' scales
out anew in theirs. Needs no GPU."""
import os
import re

import async_stage_tile_amd as pt
from tests.conftest import ROOT
from tests.test_layer_abi import P, gemm

M, N, K = 4096, 4096, 16416


def scale_bytes(rows):
    """16 bytes a row for every 512 k's."""
    return rows * -(-K // 512) * 16


def test_a_missing_or_short_one_is_refused():
    need = pt.pipe_gemm_mxfp4_workspace_bytes(M, N, K)
    assert need == scale_bytes(M) + scale_bytes(N)
    pitch = -(-(K // 32) // 16) * 16
    kw = dict(M=M, N=N, K=K, lda=K // 2, ldw=K // 2, ldsa=pitch, ldsw=pitch, ldc=N)
    assert gemm(**kw) == pt.PIPE_ERR_WORKSPACE
    assert gemm(ws=P, wsb=need - 1, **kw) == pt.PIPE_ERR_WORKSPACE
    assert gemm(ws=P + 8, wsb=need, **kw) == pt.PIPE_ERR_ALIGN


def test_the_header_names_both_uses():
    txt = open(os.path.join(ROOT, "include", "pipe_linear.h")).read()
    said = re.search(r"/\*((?:(?!\*/).)*)\*/\s*pipe_status_t pipe_gemm_mxfp4_workspace_bytes", txt, re.S).group(1)
    assert "partial products" in said and "scales" in said, said
