"""Programmatic dependent launch: a kernel that may start under the one before
it sees that kernel's writes only through its own griddepcontrol.wait.  So every
kernel that takes part waits, all of its threads, before its first use of memory:
one unconditional pdl_wait, read off the sources."""
import os
import re

import pytest

from tests.conftest import ROOT

CSRC = os.path.join(ROOT, "variable_size_expert_gb300", "csrc")


def _kernels():
    for name in sorted(os.listdir(CSRC)):
        if not name.endswith(".cu"):
            continue
        with open(os.path.join(CSRC, name)) as f:
            text = f.read()
        for m in re.finditer(r"^(?:template <[^\n]*>\n)?__global__.*?\n}\n", text, re.S | re.M):
            body = re.sub(r"//[^\n]*", "", m.group(0))
            if "pdl_trigger" in body or "pdl_wait" in body:
                yield name, re.search(r"(\w+)\s*\(\s*(?:const|float|int|void)", body).group(1), body


KERNELS = list(_kernels())


def test_kernels_were_found():
    assert len(KERNELS) >= 12


@pytest.mark.parametrize("name,kernel,body", KERNELS, ids=[f"{n}:{k}" for n, k, _ in KERNELS])
def test_every_thread_waits_first(name, kernel, body):
    waits = re.findall(r"^.*pdl_wait\(\).*$", body, re.M)
    assert len(waits) == 1, waits
    assert re.fullmatch(r"  pdl_wait\(\);\s*", waits[0]), waits[0]      # a statement of the outermost block
