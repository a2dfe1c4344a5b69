"""Tensors that a call may be given as one are not declared apart in its kernels, without a GPU.

A kernel's pointer that says __restrict__ promises that what is stored through it is loaded through no
other one.  Where the interface lets an output take an input's place, neither of the two may say so:
results would hold by the compiler's choice of registers alone.
"""
import os
import re

import pytest

import gated_delta_rule_gdn2_amd as gdn2

CSRC = os.path.join(os.path.dirname(gdn2.__file__), "csrc")


@pytest.mark.parametrize("source,kernel,names", [
    ("gdn2_rms.hip", "rms_kernel", ("residual", "h")),
    ("gdn2_rms.hip", "rms_bwd_kernel", ("dh", "dx")),
])
def test_what_may_be_one_tensor_is_not_declared_apart(source, kernel, names):
    with open(os.path.join(CSRC, source)) as f:
        text = f.read()
    (signature,) = re.findall(r"__global__[^;{]*?\b%s\(([^)]*)\)" % kernel, text)
    params = {p.split()[-1].lstrip("*"): p for p in signature.split(",")}
    for n in names:
        assert "*" in params[n] and "__restrict__" not in params[n], params[n]
