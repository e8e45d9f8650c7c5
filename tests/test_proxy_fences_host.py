"""Shared memory that passes between ordinary accesses and bulk copies: a copy
engine's write over memory that threads have used needs each of those threads'
proxy fence, then a barrier, then the copy.  Read off the sources."""
import os
import re

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "variable_size_expert_gb300", "csrc")


def test_residual_copies_into_the_staging_area():
    with open(os.path.join(CSRC, "linear.cu")) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    copies = re.findall(r"auto fetch_res = .*?\n      };\n", text, re.S)
    assert len(copies) == 1 and len(re.findall(r"tma_load_2d\(stg", text)) == 1
    fence, barrier, copy = (copies[0].find(s) for s in
                            ("fence_proxy_async_smem();", "__syncwarp();", "tma_load_2d(stg"))
    assert 0 < fence < barrier < copy
    assert "if" not in copies[0][:barrier]      # every lane
