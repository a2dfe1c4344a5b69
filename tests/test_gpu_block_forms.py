"""The kernel forms that only large calls of the state space block take, held to the fp64 oracle.

Which form runs is a matter of sizes: two heads of 64 columns a workgroup from 512 heads of
sequences or segments on, whole heads of 128 columns from 129 on (fewer go in halves), sequences cut
into segments with and without a pass that joins them, a step past the caches above 128 MB of
states, the convolution's runs of 16 tokens from 2^17 threads on.  The bars are those of
tests/test_gpu_block.py; sequences are independent, so a few of each call are checked whole."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn2_amd as gdn2
from gated_delta_rule_gdn2_amd import block
from tests.parity_util import say
from tests.test_gpu_block import (BF16, F32, U, check_scan, conv_case, conv_ref, dev, f64, oracle_scan, packed_case, scan_case,
                                  within)

pytestmark = pytest.mark.gpu
TOKENS = ("x", "dt", "B", "C")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn2._load()


def sequence(k, n):
    """Sequence n of a case of whole sequences, as a case of one."""
    one = {m: (v[n:n + 1] if m in TOKENS else v) for m, v in k.items()}
    one["s0"] = None if k["s0"] is None else k["s0"][n:n + 1]
    return one


def part(k, cu, n):
    """Sequence n of a packed case, as a case of one."""
    one = {m: (v[None, int(cu[n]):int(cu[n + 1])] if m in TOKENS else v) for m, v in k.items()}
    one["s0"] = None if k["s0"] is None else k["s0"][n:n + 1]
    return one


def args_of(d):
    return d["x"], d["dt"], d["B"], d["C"], d["A"]


# ---- scan -----------------------------------------------------------------------------------

FORMS = [  # dtype, B, T, H, G, dk, dv, cut
    # pairs of heads of 64 columns: whole sequences, few segments, many segments
    (BF16, 16, 200, 32, 2, 128, 64, False),
    (F32, 16, 200, 32, 2, 64, 64, False),
    (BF16, 4, 1500, 32, 2, 128, 64, True),
    (BF16, 2, 2000, 32, 2, 128, 64, True),
    (F32, 4, 700, 32, 2, 64, 64, True),
    (F32, 4, 700, 32, 4, 128, 64, True),
    # heads of 128 columns in one workgroup
    (BF16, 4, 1500, 16, 1, 128, 128, True),
    (BF16, 2, 2300, 24, 2, 128, 128, True),
    (F32, 9, 70, 16, 1, 128, 128, False),
    (F32, 2, 700, 24, 2, 128, 128, True),
]


@pytest.mark.parametrize("dtype,B,T,H,G,dk,dv,cut", FORMS)
def test_scan_forms_match_oracle(dtype, B, T, H, G, dk, dv, cut):
    say("case: scan form %s B%d T%d H%d G%d dk%d dv%d" % (dtype, B, T, H, G, dk, dv))
    k = scan_case(dtype, (B, T), H, G, dk, dv, 100 + T + H + dk, B, strong=T % 200 == 100)
    assert (gdn2.ssm_fwd_workspace_bytes(B, T, H, dk, dv, dtype) > 0) == cut
    d = dev(k)
    y, s = gdn2.ssm_fwd(*args_of(d), d["D"], d["dt_bias"], d["s0"])
    for n in sorted({0, B // 2, B - 1}):
        one = sequence(k, n)
        check_scan(one, y[n:n + 1], s[n:n + 1], oracle_scan(one), (T + 63) // 64)
    state = d["s0"].clone()
    y2, _ = gdn2.ssm_fwd(*args_of(d), d["D"], d["dt_bias"], state, final_state=state)
    assert torch.equal(y, y2) and torch.equal(s, state)


PACKED = [  # dtype, lengths, H, G, dk, dv, cut
    (BF16, [90, 64, 1, 0, 130, 63, 200, 5] * 3, 32, 2, 128, 64, True),
    (BF16, [700, 0, 300, 2300, 1, 64, 257, 40] + [9] * 8, 32, 2, 128, 64, True),
    (F32, [500, 1, 900, 0, 65, 128], 32, 2, 64, 64, True),
    (BF16, [600, 1100, 0, 257, 2, 500], 32, 2, 128, 128, True),
    (BF16, [40, 65, 128, 0, 3, 17, 1, 9, 30], 16, 1, 64, 128, True),
    (F32, [500, 1, 400, 0, 65, 130], 24, 2, 128, 128, True),
    (F32, [20, 30, 1, 0, 40, 9, 8, 3, 7], 16, 1, 128, 128, False),
]


@pytest.mark.parametrize("dtype,lengths,H,G,dk,dv,cut", PACKED)
def test_packed_scan_forms_match_oracle(dtype, lengths, H, G, dk, dv, cut):
    say("case: packed form %s N%d H%d G%d dk%d dv%d" % (dtype, len(lengths), H, G, dk, dv))
    k, cu = packed_case(dtype, lengths, H, G, dk, dv, 300 + sum(lengths), lead=2, behind=3)
    assert (gdn2.ssm_fwd_varlen_workspace_bytes(len(lengths), k["x"].shape[0], H, dk, dv, dtype) > 0) == cut
    d = dev(k)
    y0 = torch.full_like(d["x"], 7.0)
    y, s = gdn2.ssm_fwd_varlen(*args_of(d), cu.cuda(), d["D"], d["dt_bias"], d["s0"], y=y0)
    assert (y[:2] == 7).all() and (y[int(cu[-1]):] == 7).all()
    for n, length in enumerate(lengths):
        if length == 0:
            assert torch.equal(s[n].cpu(), k["s0"][n])
        elif n < 8:
            one = part(k, cu, n)
            check_scan(one, y[None, int(cu[n]):int(cu[n + 1])], s[n:n + 1], oracle_scan(one), (length + 63) // 64)
    state = d["s0"].clone()
    y2, _ = gdn2.ssm_fwd_varlen(*args_of(d), cu.cuda(), d["D"], d["dt_bias"], state, y=torch.full_like(y, 7.0),
                                final_state=state)
    assert torch.equal(y, y2) and torch.equal(s, state)
