"""The bounds-checked debug build on the paged cache's cases: pages, rows, parts
and slabs outside their extents would be recorded (SPEC_ERR_DEVICE_BOUNDS).  One
fresh process that loads the checked library; results are held to the oracle as
in the normal build."""
import os
import re
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_54_gb300", "csrc")

_CHILD = r"""
import sys
sys.path.insert(0, sys.argv[1])
import numpy as np, torch
import speculative_decoding_verification_54_gb300 as sv
from speculative_decoding_verification_54_gb300 import _build
sv.load(_build.build(checked=True))
torch.cuda.set_device(0)
from tests import test_gpu_paged as t
n = 0
for c in t.APPEND:
    t.test_append(sv, *c)
    n += 1
t.test_append_many_sequences(sv)
for c in t.ATTEND:
    t.test_attention(sv, *c)
    n += 1
for c in (t.LARGE[1], t.LARGE[3], t.LARGE[4]):  # split items, a mask, row blocks
    t.test_attention_large(sv, *c)
    n += 1
t.test_pages_and_lengths_out_of_range_are_reported(sv)
from tests import test_gpu_paged_hidden as h  # rows that the join sums again
for c in h.SHAPES[2:4]:
    h.test_new_entries(sv, c, "last")
print("ok", n)
"""


@pytest.mark.gpu
def test_checked_build_of_the_paged_calls():
    r = subprocess.run([sys.executable, "-c", _CHILD, ROOT], cwd=ROOT, capture_output=True, text=True, timeout=600)
    assert r.returncode == 0, r.stderr[-3000:]
    assert r.stdout.startswith("ok"), r.stdout[-2000:]


@pytest.mark.parametrize("name,least", [("attend.cuh", 8), ("kvappend.cuh", 4)])
def test_the_kernels_check_their_computed_indices(name, least):
    text = open(os.path.join(CSRC, name), encoding="utf-8").read()
    assert len(re.findall(r"\bin_bounds\(", re.sub(r"//.*", "", text))) >= least
