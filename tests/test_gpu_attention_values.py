"""GPU tests of attention at values that seldom occur: scores that outgrow a reference, infinities in a
step's own token, values near fp32's end.  Bars as derived in test_gpu_attention."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn2_amd as gdn2
from oracle import attention as A
from tests.parity_util import say
from tests.test_gpu_attention import BF16, F32, INF, MANY, NAN, U, check_fwd, f64, fwd, half_step, pieces, within

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


# ---- values near the end of fp32 ------------------------------------------------------------

def check(q, k, v, o, lse):
    """check_fwd but for the channel of tiny values, which rows of large ones may lose."""
    keep = [c for c in range(v.shape[-1]) if c != 5]
    ro, rl = A.attention(q, k, v)
    s, seen, off, top = pieces(q, k, None, None)
    p = np.where(seen, np.exp(np.where(seen, s, 0.0) - rl.T[..., None]), 0.0)
    n, r = seen.sum(-1, keepdims=True) + 8, half_step(q.dtype)
    va = np.abs(np.repeat(f64(v), q.shape[1] // k.shape[1], 1))
    spread = (p * (off + n * U)).sum(-1)
    tol = np.einsum("hts,shd->thd", p * (off + r + n * U), va) + np.abs(ro) * spread.T[..., None] + r * np.abs(ro)
    within("o", o[..., keep], ro[..., keep], tol[..., keep])
    within("lse", lse, rl, spread.T + 8 * U * (1 + np.abs(rl) + top[..., 0].T))


BIG = [  # T, S, H, G, d
    (300, 300, 2, 1, 64), (300, 300, 2, 1, 128), (6, 3001, 4, 2, 64), (40, 5000, 1, 1, 128), (2100, 2130, 1, 1, 128)]


@MANY
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("T,S,H,G,d", BIG)
def test_finite_values_give_finite_outputs(dtype, T, S, H, G, d, many):
    """Values up to 2^126 behind scores that grow along the keys, so that the reference stays behind: outputs
    are means of values and stay below the largest.  Other channels keep their bits, and queries that see none of
    the large values keep them in all, those of tiny values too."""
    if many and S > 3001:
        pytest.skip("the same form as the fewer")
    say("case: large values %s T%d S%d d%d" % (dtype, T, S, d))
    g = torch.Generator("cpu").manual_seed(S + d)
    q, k, v = (torch.randn(1, n, h, d, generator=g) for n, h in ((T, H), (S, G), (S, G)))
    q[..., 0], k[..., 0] = 1.0, torch.linspace(0, 40, S)[None, :, None]  # a weight grows by up to e^5 in all
    v[..., 5] *= 2.0 ** -100
    q, k, v = (x.to(dtype) for x in (q, k, v))
    o, lse = fwd(many, q.cuda(), k.cuda(), v.cuda())
    rest = [c for c in range(d) if c not in (3, 4, 5)]
    for size, first in ((2.0 ** 105, 0), (2.0 ** 126, 0), (2.0 ** 126, S - 3 * T // 4)):
        big = v.float().clone()
        big[:, first:, :, 3] = size * torch.rand(1, S - first, G, generator=g)
        big[:, first:, :, 4] = size
        big = big.to(dtype)
        o2, lse2 = fwd(many, q.cuda(), k.cuda(), big.cuda())
        check(q[0], k[0], big[0], o2[0], lse2[0])
        assert torch.equal(lse, lse2)
        assert torch.equal(o[..., rest], o2[..., rest])
        blind = max(0, first - (S - T))
        assert torch.equal(o[:, :blind], o2[:, :blind])
