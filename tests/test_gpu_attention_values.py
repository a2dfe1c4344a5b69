"""GPU tests of attention at values that seldom occur: scores that outgrow a reference.  Bars as derived in test_gpu_attention."""
import pytest
import torch

import gated_delta_rule_gdn2_amd as gdn2
from tests.parity_util import say
from tests.test_gpu_attention import BF16, F32, MANY, check_fwd, fwd

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn2._load()


# ---- the reference of the softmax -----------------------------------------------------------

@MANY
@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)])
def test_a_neighbours_scores_change_no_bit(dtype, d, many):
    """Query 400 meets two keys of weight e^8 in one tile, one in each half of the lanes that hold its scores
    (keys 4 apart of 8): each half stays below 2^12, their sum does not.  Whether query 401, of the same wave,
    outgrows its own reference at that tile changes no bit of it."""
    say("case: two heavy halves %s d%d" % (dtype, d))
    T = 512
    g = torch.Generator("cpu").manual_seed(d)
    q, k, v = torch.zeros(1, T, 1, d), torch.zeros(1, T, 1, d), torch.randn(1, T, 1, d, generator=g)
    k[0, :, 0, 0] = torch.rand(T, generator=g) * 0.125
    k[0, 320, 0, 0] = k[0, 324, 0, 0] = 8.125  # e^8 = 2981 above the others' largest
    k[0, 320, 0, 1] = 16.0
    q[0, 400, 0, 0] = 1.0
    q, k, v = (x.to(dtype) for x in (q, k, v))
    o, lse = fwd(many, q.cuda(), k.cuda(), v.cuda(), scale=1.0)
    check_fwd(q[0], k[0], v[0], o[0], lse[0], None, 1.0)
    loud = q.clone()
    loud[0, 401, 0, 1] = 1.0
    o2, lse2 = fwd(many, loud.cuda(), k.cuda(), v.cuda(), scale=1.0)
    check_fwd(loud[0], k[0], v[0], o2[0], lse2[0], None, 1.0)
    others = torch.arange(T) != 401
    assert torch.equal(o[0, others], o2[0, others]) and torch.equal(lse[0, others], lse2[0, others])
