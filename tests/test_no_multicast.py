"""No copy or barrier of the library is delivered to several CTAs of a cluster at once: processes on several GPUs load the
same library, and cluster multicast may stand only in code that one GPU runs alone. CTAs share through stores and bulk copies
into each other's shared memory."""
import glob
import os
import re

import pytest

import bench

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "sparse_mla_attention_04_gb300", "csrc")


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*"))), ids=os.path.basename)
def test_sources_hold_no_multicast(path):
    code = bench._code_only(open(path, encoding="utf-8").read())
    assert not re.search(r"multicast|multimem", code, re.I)
