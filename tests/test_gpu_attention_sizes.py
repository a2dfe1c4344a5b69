"""GPU tests of attention at counts of sequences and heads that do not divide into the XCDs."""
import pytest
import torch

import gated_delta_rule_gdn2_amd as gdn2
from oracle import attention as A
from tests.parity_util import say
from tests.test_gpu_attention import BF16, F32, U, case, check_bwd, check_fwd, f64, first_of, rotary_bar, times, within

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn2._load()


@pytest.mark.parametrize("dtype,B,T,H,G,d", [
    (BF16, 67, 130, 3, 1, 64), (BF16, 65, 300, 3, 3, 128), (BF16, 1025, 5, 1, 1, 64), (BF16, 333, 129, 6, 2, 128), (BF16, 21, 1100, 5, 5, 64),
    (F32, 67, 130, 3, 1, 64), (F32, 129, 70, 3, 3, 128), (BF16, 9, 351, 16, 1, 128)])
def test_counts_that_do_not_divide(dtype, B, T, H, G, d):
    """One sequence B times: every copy has the same bits, and the first is right."""
    say("case: copies %s B%d T%d H%d G%d d%d" % (dtype, B, T, H, G, d))
    q, k, v, g = case(dtype, T, T, H, G, d, B + T)
    dev = [times(B, x.cuda()) for x in (q, k, v)]
    o, lse = gdn2.attn_fwd(*dev)
    grads = gdn2.attn_bwd(times(B, g.cuda()), *dev, o, lse)
    firsts = first_of(B, o, lse, *grads.values())
    check_fwd(q[0], k[0], v[0], firsts[0][0], firsts[1][0])
    check_bwd(g[0], q[0], k[0], v[0], firsts[0][0], firsts[1][0], dict(zip(grads, (x[0] for x in firsts[2:]))))


def test_a_million_sequences_of_one_token():
    """Each query sees its own key alone: o is its value, dv the sum over the heads' d_o, which three roundings
    of a weight of one do not change in bf16."""
    B, H, d = (1 << 20) + 1, 2, 64
    if torch.cuda.mem_get_info()[0] < 8 << 30:
        pytest.skip("needs 8 GB")
    g = torch.Generator("cuda").manual_seed(2)
    q, k, v, d_o = (torch.randn(B, 1, h, d, generator=g, device="cuda", dtype=torch.float32).to(BF16) for h in (H, 1, 1, H))
    o, lse = gdn2.attn_fwd(q, k, v)
    assert torch.equal(o, v.expand_as(o))
    scores = (q.float() * k.float()).sum(-1) / 8
    assert ((lse - scores).abs() <= 1e-5 * (1 + scores.abs())).all()  # 64 products' roundings and the logarithm's
    grads = gdn2.attn_bwd(d_o, q, k, v, o, lse)
    want = (d_o[:, :, :1].float() + d_o[:, :, 1:].float()).to(BF16)
    assert torch.equal(grads["dv"], want)
    cu = torch.arange(257, dtype=torch.int64, device="cuda")
    part, _ = gdn2.attn_fwd_varlen(q[:256, 0], k[:256, 0], v[:256, 0], cu)
    assert torch.equal(part, o[:256, 0])


@pytest.mark.parametrize("window", [None, 20, (1 << 63) - 1])
def test_step_at_the_last_position(window):
    """Position 2^63 - 1 and the ones before it see as many tokens as any other."""
    C, H, G, d = 50, 2, 1, 64
    last = (1 << 63) - 1
    places = [last, last - 1, last - 25, 3]
    g = torch.Generator("cpu").manual_seed(8)
    q, k, v, kc, vc = (torch.randn(s, generator=g).to(BF16) for s in ((4, H, d), (4, G, d), (4, G, d), (4, C, G, d), (4, C, G, d)))
    k2, v2 = kc.cuda(), vc.cuda()
    o = gdn2.attn_step(q.cuda(), k.cuda(), v.cuda(), k2, v2, torch.tensor(places, device="cuda"), window=window)
    for i, p in enumerate(places):
        kc[i, p % C], vc[i, p % C] = k[i], v[i]
        tokens = [t % C for t in range(max(0, p + 1 - min(C, window or C)), p + 1)]
        check_fwd(q[i:i + 1], kc[i, tokens], vc[i, tokens], o[i:i + 1], None)
    assert torch.equal(k2.cpu(), kc) and torch.equal(v2.cpu(), vc)


@pytest.mark.parametrize("tokens,H,d", [((1 << 27) - 8, 1, 2), ((1 << 25) - 8, 7, 32)])
def test_rotary_of_the_most_tokens(tokens, H, d):
    """The first and the last tokens: angles of 2^27 radians are off by 2^-51 of themselves, 2^-24."""
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB")
    g = torch.Generator("cuda").manual_seed(3)
    q = torch.empty(tokens, H, d, device="cuda")
    for at in (slice(0, 500), slice(tokens - 500, tokens)):
        q[at] = torch.randn(500, H, d, generator=g, device="cuda")
    freq = gdn2.rotary_frequencies(2)
    out, _ = gdn2.rotary(q, None, freq.cuda())
    for at in (slice(0, 500), slice(tokens - 500, tokens)):
        x = q[at].cpu()
        ref = A.rotary(x, freq, range(tokens)[at])
        pair = abs(f64(x))[..., :2].sum(-1, keepdims=True)
        within("q", out[at], ref, rotary_bar(x, freq, False) + U * pair)
