"""GPU tests of attention at values that seldom occur: scores that outgrow a reference, infinities in a
step's own token.  Bars as derived in test_gpu_attention."""
import pytest
import torch

import gated_delta_rule_gdn2_amd as gdn2
from tests.parity_util import say
from tests.test_gpu_attention import BF16, F32, INF, MANY, NAN, check_fwd, fwd

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


# ---- infinities in a step's own token -------------------------------------------------------

@pytest.mark.parametrize("dtype,d", [(BF16, 64), (BF16, 128), (F32, 64), (F32, 128)])
@pytest.mark.parametrize("bad", [INF, -INF, NAN])
@pytest.mark.parametrize("C,window", [(200, None), (3000, None), (200, 33)])
def test_step_with_values_that_are_not_finite(dtype, d, bad, C, window):
    """The newest token's value, or an older one's, in one channel: that channel alone shows it, whether the
    tokens seen fill their tiles of 32 or not."""
    say("case: step, %s in a value, %s d%d C%d window %s" % (bad, dtype, d, C, window))
    H, G = 4, 2
    places = [0, 1, 30, 31, 32, 63, 100, 159, 199, 200, 2047, 2999, 3100]
    n = len(places)
    g = torch.Generator("cuda").manual_seed(C + d)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    q, k, v, kc, vc = r(n, H, d), r(n, G, d), r(n, G, d), r(n, C, G, d), r(n, C, G, d)
    at = torch.tensor(places, device="cuda")
    clean = gdn2.attn_step(q, k, v, kc.clone(), vc.clone(), at, window=window)
    assert torch.isfinite(clean).all()
    dirty = v.clone()
    dirty[:, 1, 5] = bad
    o = gdn2.attn_step(q, k, dirty, kc.clone(), vc.clone(), at, window=window)
    hit = torch.zeros(n, H, d, dtype=torch.bool, device="cuda")
    hit[:, H // G:, 5] = True
    assert torch.equal(o[~hit], clean[~hit])
    same = torch.isnan(o[hit]) if bad != bad else o[hit] == bad
    assert same.all(), [places[i] for i in range(n) if not same.view(n, -1)[i].all()]
    # an older token's: the one before the newest, where there is one that is seen
    older = vc.clone()
    for i, p in enumerate(places):
        older[i, (p - 1) % C, 0, 7] = bad
    o = gdn2.attn_step(q, k, v, kc.clone(), older, at, window=window)
    hit = torch.zeros(n, H, d, dtype=torch.bool, device="cuda")
    hit[[i for i, p in enumerate(places) if p > 0], :H // G, 7] = True
    assert torch.equal(o[~hit], clean[~hit])
    assert (torch.isnan(o[hit]) if bad != bad else o[hit] == bad).all()
