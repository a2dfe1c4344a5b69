"""GPU parity of the attention block with its fp64 oracle.

Bars, element by element, from the arithmetic (u = 2^-24, the half step of fp32; r = 2^-8, that of
bf16, or 0 for fp32 inputs):

* a score is a sum of d products: off by (d + 4) u A, A the sum of absolute values times the scale;
  in the exponent it is multiplied by a rounded constant and meets a rounded reference of the size of
  the row's scores, 4 u (|s| + M), M the largest |s| the row sees.  A weight is then off by
  D = (d + 4) u A + 4 u (|s| + M) + 4 u of itself (the exponential 1 ulp, the sum's terms scaled).
* o: sum P |v| (D + r + (n + 8) u) + |o| sum P (D + (n + 8) u), n the keys, and r |o| on the store:
  the weights enter the second product rounded, the sum unrounded.  lse: sum P (D + (n + 8) u) +
  8 u (1 + |lse| + M).
* gradients: dP and delta are sums of d products, off by (d + 4) u of their absolute sums B and C, so
  dS by E = P (D |dP - delta| + (d + 4) u (B + C) + 2 u |dP - delta|) + r |dS|; each gradient by
  the sum of E (or P (D + r)) times the absolute other factor, (n + 8) u of the absolute sum (n its
  terms), and r of itself.  D here has |lse| for M, which is given.
* rotary: a part of a turn is off by 2^-25, 3.2 u radians; sine and cosine by 2 ulp (4 u), three
  roundings follow: 12 u (|a| + |b|), and r |y|.
* norm: a row's sum passes at most 96 roundings, so rstd is off by 52 u of itself, y by 56 u + r,
  h by u + r; sums over rows at most 600 roundings; 8 bits: half a step of e4m3, 2^-4 of the
  value or 2^-10 of the scale, whichever is more."""
import math

import numpy as np
import pytest
import torch

import gated_delta_rule_gdn2_amd as gdn2
from oracle import attention as A
from tests.parity_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn2._load()


def f64(t):
    return t.detach().cpu().double().numpy()


def half_step(dtype):
    return 2.0 ** -8 if dtype == BF16 else 0.0


def within(name, got, ref, tol):
    got = f64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    fine = np.isfinite(ref)
    assert np.array_equal(got[~fine], ref[~fine], equal_nan=True), name
    assert np.isfinite(got[fine]).all(), name
    bar = np.broadcast_to(tol, ref.shape)[fine] + 1e-30
    worst = float((np.abs(got[fine] - ref[fine]) / bar).max()) if fine.any() else 0.0
    say("  %-8s worst %.3f of its bar" % (name, worst))
    assert worst <= 1.0, (name, worst)


# ---- attention ------------------------------------------------------------------------------

def case(dtype, Tq, S, H, G, d, seed, B=1, spread=1.0):
    g = torch.Generator("cpu").manual_seed(seed)
    r = lambda *s: (torch.randn(s, generator=g) * spread).to(dtype)
    return r(B, Tq, H, d), r(B, S, G, d), r(B, S, G, d), r(B, Tq, H, d)


def pieces(q, k, window, scale, lse=None):
    """Of one sequence, [H,T,S]: scores, weights and what a weight may be off by."""
    d = q.shape[-1]
    q, k = f64(q), f64(k)
    share = q.shape[1] // k.shape[1]
    scale = d ** -0.5 if scale is None else scale
    s = A.scores(q, k, window, scale)
    seen = np.isfinite(s)
    a = np.einsum("thd,shd->hts", np.abs(q), np.abs(np.repeat(k, share, 1))) * scale
    s0 = np.where(seen, s, 0.0)
    top = np.abs(s0).max(-1, keepdims=True, initial=0.0) if lse is None else np.abs(np.where(np.isfinite(lse), lse, 0.0)).T[..., None]
    off = ((d + 4) * a + 4 * (np.abs(s0) + top) + 4) * U
    return s, seen, off, top


def check_fwd(q, k, v, o, lse, window=None, scale=None):
    """One sequence's tensors [T,...]."""
    dtype, share = q.dtype, q.shape[1] // k.shape[1]
    ro, rl = A.attention(q, k, v, window, scale)
    s, seen, off, top = pieces(q, k, window, scale)
    p = np.where(seen, np.exp(np.where(seen, s, 0.0) - np.where(np.isfinite(rl), rl, 0.0).T[..., None]), 0.0)
    n = seen.sum(-1, keepdims=True) + 8
    r = half_step(dtype)
    va = np.abs(np.repeat(f64(v), share, 1))
    spread = (p * (off + n * U)).sum(-1)
    tol = np.einsum("hts,shd->thd", p * (off + r + n * U), va) + np.abs(ro) * spread.T[..., None] + r * np.abs(ro)
    within("o", o, ro, tol)
    if lse is not None:
        within("lse", lse, rl, spread.T + 8 * U * (1 + np.abs(np.where(np.isfinite(rl), rl, 0.0)) + top[..., 0].T))


def check_bwd(d_o, q, k, v, o, lse, grads, window=None, scale=None):
    dtype, share, d = q.dtype, q.shape[1] // k.shape[1], q.shape[-1]
    ref = A.attention_bwd(d_o, q, k, v, o, lse, window, scale)
    sc = d ** -0.5 if scale is None else scale
    l64 = f64(lse)
    s, seen, off, _ = pieces(q, k, window, scale, l64)
    p = np.where(seen, np.exp(np.where(seen, s, 0.0) - np.where(np.isfinite(l64), l64, 0.0).T[..., None]), 0.0)
    r = half_step(dtype)
    g, qq, oo = f64(d_o), f64(q), f64(o)
    kk, vv = np.repeat(f64(k), share, 1), np.repeat(f64(v), share, 1)
    gap = np.einsum("thd,shd->hts", g, vv) - (g * oo).sum(-1).T[..., None]
    sums = np.einsum("thd,shd->hts", np.abs(g), np.abs(vv)) + (np.abs(g) * np.abs(oo)).sum(-1).T[..., None]
    ds = np.abs(p * gap)
    e = p * (off * np.abs(gap) + (d + 4) * U * sums + 2 * U * np.abs(gap)) + r * ds
    S, G = k.shape[:2]
    fold = lambda x: x.reshape(S, G, share, d).sum(2)
    nq, nk = (seen.sum(-1, keepdims=True) + 8) * U, (seen.sum(1, keepdims=True) * share + 8) * U
    tq = sc * np.einsum("hts,shd->thd", e + nq * ds, np.abs(kk))
    tk = sc * fold(np.einsum("hts,thd->shd", e + nk * ds, np.abs(qq)))
    tv = fold(np.einsum("hts,thd->shd", p * (off + r + nk), np.abs(g)))
    for name, x, t in zip(("dq", "dk", "dv"), ref, (tq, tk, tv)):
        within(name, grads[name], x, t + (r + 2 * U) * np.abs(x))


# Few workgroups share their rows between waves and are taken in parts; the same sequences many times over
# are not.  Every copy of a sequence has the same bits.
MANY = pytest.mark.parametrize("many", [False, True], ids=["few", "many"])


def copies(many, q, k):
    """Copies of the sequences q [B,T,H,d], k [B,S,G,d] that make more than 4096 blocks of 32 rows."""
    (B, T, H, _), (_, S, G, _) = q.shape, k.shape
    return 1 + 4096 // max(1, B * min(-(-T // 32) * H, -(-S // 32) * G)) if many else 1


def first_of(n, *outs):
    firsts = []
    for x in outs:
        B = x.shape[0] // n
        bits = x.view(torch.int16 if x.dtype == BF16 else torch.int32).reshape(n, -1)
        assert (bits == bits[:1]).all()
        firsts.append(x[:B])
    return firsts


def times(n, x):
    return x.repeat(n, *[1] * (x.dim() - 1)) if n > 1 else x


def fwd(many, q, k, v, **kw):
    n = copies(many, q, k)
    return first_of(n, *gdn2.attn_fwd(*[times(n, x) for x in (q, k, v)], **kw))


def bwd(many, d_o, q, k, v, o, lse, **kw):
    n = copies(many, q, k)
    grads = gdn2.attn_bwd(*[times(n, x) for x in (d_o, q, k, v, o, lse)], **kw)
    return dict(zip(grads, first_of(n, *grads.values())))


FWD = [  # dtype, B, T, S, H, G, d, window
    (BF16, 1, 1, 1, 1, 1, 64, None), (F32, 1, 1, 1, 2, 1, 128, None),
    (BF16, 2, 1, 77, 8, 2, 128, None), (BF16, 1, 31, 31, 2, 2, 64, None), (BF16, 2, 33, 33, 6, 2, 128, None),
    (BF16, 1, 64, 64, 2, 1, 64, None), (BF16, 1, 65, 65, 3, 1, 128, 1), (BF16, 2, 127, 127, 4, 4, 64, 31), (BF16, 1, 128, 128, 2, 1, 128, 64),
    (BF16, 1, 129, 129, 2, 1, 128, 65), (BF16, 1, 200, 333, 4, 2, 64, None), (BF16, 1, 300, 300, 2, 1, 128, 100),
    (BF16, 1, 520, 520, 2, 1, 64, 256), (BF16, 1, 90, 40, 2, 1, 128, None), (BF16, 1, 300, 5, 2, 2, 64, 3), (BF16, 1, 5, 2500, 2, 1, 64, None),
    (BF16, 1, 3, 1100, 20, 1, 128, 700), (BF16, 1, 40, 0, 2, 1, 64, None), (BF16, 17, 9, 9, 2, 1, 128, None),
    (F32, 1, 33, 33, 2, 1, 64, None), (F32, 2, 65, 100, 4, 2, 128, 40), (F32, 1, 130, 130, 2, 2, 64, 33), (F32, 1, 70, 20, 2, 1, 128, None),
    (F32, 1, 4, 1500, 2, 1, 128, None), (F32, 1, 257, 257, 1, 1, 64, None),
]


@MANY
@pytest.mark.parametrize("dtype,B,T,S,H,G,d,window", FWD)
def test_forward_matches_oracle(dtype, B, T, S, H, G, d, window, many):
    say("case: forward %s B%d T%d S%d H%d G%d d%d window %s" % (dtype, B, T, S, H, G, d, window))
    q, k, v, _ = case(dtype, T, S, H, G, d, 7 * T + S, B)
    dev = [x.cuda() for x in (q, k, v)]
    o, lse = fwd(many, *dev, window=window)
    torch.cuda.synchronize()
    for b in range(B):
        check_fwd(q[b], k[b], v[b], o[b], lse[b], window)
    again, lse2 = fwd(many, *dev, window=window)
    assert torch.equal(o, again) and torch.equal(lse, lse2)
    if many:
        return
    only, none = gdn2.attn_fwd(*dev, window=window, stats=False)
    assert none is None and torch.equal(only, o)


@MANY
@pytest.mark.parametrize("dtype,T,S,H,G,d,window", [c[:1] + c[2:] for c in FWD if c[3]] + [
    (BF16, 96, 96, 4, 1, 128, 96), (BF16, 260, 260, 4, 2, 128, 130), (F32, 100, 160, 6, 2, 64, 50), (BF16, 600, 620, 8, 1, 64, None),
    (BF16, 530, 530, 12, 2, 128, 400), (F32, 410, 410, 4, 1, 128, None), (F32, 300, 333, 8, 1, 64, 250)])
def test_gradients_match_oracle(dtype, T, S, H, G, d, window, many):
    say("case: gradients %s T%d S%d H%d G%d d%d window %s" % (dtype, T, S, H, G, d, window))
    q, k, v, g = case(dtype, T, S, H, G, d, 3 * T + S)
    o, lse = A.attention(q[0], k[0], v[0], window)
    o, lse = torch.from_numpy(o).to(dtype)[None], torch.from_numpy(lse).float()[None]
    dev = [x.cuda() for x in (g, q, k, v, o, lse)]
    grads = bwd(many, *dev, window=window)
    torch.cuda.synchronize()
    check_bwd(g[0], q[0], k[0], v[0], o[0], lse[0], {n: x[0] for n, x in grads.items()}, window)
    again = bwd(many, *dev, window=window)
    assert all(torch.equal(grads[n], again[n]) for n in grads)


@pytest.mark.parametrize("dtype,scale", [(BF16, 0.03), (F32, 1.7)])
def test_scale_and_large_scores(dtype, scale):
    q, k, v, g = case(dtype, 70, 70, 2, 1, 64, 5, spread=2.0)
    o, lse = gdn2.attn_fwd(q.cuda(), k.cuda(), v.cuda(), scale=scale)
    check_fwd(q[0], k[0], v[0], o[0], lse[0], None, scale)
    grads = gdn2.attn_bwd(g.cuda(), q.cuda(), k.cuda(), v.cuda(), o, lse, scale=scale)
    check_bwd(g[0], q[0], k[0], v[0], o[0], lse[0], {n: x[0] for n, x in grads.items()}, None, scale)


@pytest.mark.parametrize("d", [64, 128])
def test_gradients_against_differences(d):
    """A direction's slope of sum(d_o * o) in fp32, from calls of the forward pass alone."""
    q, k, v, g = (x.cuda() for x in case(F32, 75, 90, 4, 2, d, 17))
    o, lse = gdn2.attn_fwd(q, k, v, window=40)
    grads = gdn2.attn_bwd(g, q, k, v, o, lse, window=40)
    gen = torch.Generator("cuda").manual_seed(3)
    h = 2.0 ** -6
    for name, at in (("dq", 0), ("dk", 1), ("dv", 2)):
        args = [q, k, v]
        way = torch.randn(args[at].shape, generator=gen, device="cuda")
        values = []
        for sign in (1, -1):
            moved = list(args)
            moved[at] = args[at] + sign * h * way
            values.append((g.double() * gdn2.attn_fwd(*moved, window=40)[0].double()).sum().item())
        slope, want = (values[0] - values[1]) / (2 * h), (grads[name].double() * way.double()).sum().item()
        # the difference's own error: h^2 / 6 of a third derivative, and fp32 outputs' roundings / h
        size = (grads[name].double().abs() * way.double().abs()).sum().item()
        assert abs(slope - want) <= 4 * h * h * size + 1e-4 * size, (name, slope, want)


def parts(qkv, H, G, d):
    q, k, v = qkv.split((H * d, G * d, G * d), -1)
    return q.unflatten(-1, (H, d)), k.unflatten(-1, (G, d)), v.unflatten(-1, (G, d))


@pytest.mark.parametrize("dtype,H,G,d", [(BF16, 4, 2, 64), (F32, 2, 1, 128)])
def test_parts_of_one_tensor(dtype, H, G, d):
    g = torch.Generator("cpu").manual_seed(2)
    qkv = torch.randn(2, 150, (H + 2 * G) * d + 16, generator=g).to(dtype).cuda()
    q, k, v = parts(qkv[..., :(H + 2 * G) * d], H, G, d)
    o, lse = gdn2.attn_fwd(q, k, v, window=70)
    o2, lse2 = gdn2.attn_fwd(q.contiguous(), k.contiguous(), v.contiguous(), window=70)
    assert torch.equal(o, o2) and torch.equal(lse, lse2)
    d_o = torch.randn(o.shape, generator=g).to(dtype).cuda()
    a = gdn2.attn_bwd(d_o, q, k, v, o, lse, window=70)
    b = gdn2.attn_bwd(d_o, q.contiguous(), k.contiguous(), v.contiguous(), o, lse, window=70)
    assert all(torch.equal(a[n], b[n]) and a[n].is_contiguous() for n in a)


def offsets(lengths):
    return torch.tensor([0] + list(np.cumsum(lengths)), dtype=torch.int64)


PACKED = [  # dtype, query lengths, keys before them, H, G, d, window
    (BF16, [5, 0, 130, 1, 64, 33], None, 4, 2, 64, None),
    (BF16, [129, 257, 1], None, 2, 1, 128, 100),
    (BF16, [7, 65, 0, 128], [200, 0, 50, 31], 4, 1, 128, None),
    (BF16, [3, 1, 2], [700, 1500, 0], 2, 2, 64, 900),
    (BF16, [300, 40, 1], None, 8, 1, 64, None), (BF16, [9, 190, 64], [70, 0, 3], 12, 2, 128, 150),
    (F32, [40, 0, 1, 100], None, 2, 1, 64, 30),
    (F32, [20, 66], [90, 3], 2, 1, 128, None),
]


@MANY
@pytest.mark.parametrize("dtype,lengths,past,H,G,d,window", PACKED)
def test_packed_matches_oracle(dtype, lengths, past, H, G, d, window, many):
    say("case: packed %s %s after %s H%d G%d d%d window %s" % (dtype, lengths, past, H, G, d, window))
    n = len(lengths)
    keys = [a + b for a, b in zip(lengths, past or [0] * n)]
    tail = 9  # tokens of no sequence
    R = 2 + (8192 if d == 64 else 1024) // (n * G) if many else 1  # the sequences so many times
    cu, cu_k = offsets(lengths * R), offsets(keys * R)
    q, _, _, g = case(dtype, sum(lengths) + tail, 1, H, G, d, 11)
    _, k, v, _ = case(dtype, 1, sum(keys) + tail, H, G, d, 12)
    q, k, v, g = (x[0] for x in (q, k, v, g))
    # what lies behind the last sequence is nobody's: it may be anything
    for x, end in ((q, sum(lengths)), (k, sum(keys)), (v, sum(keys)), (g, sum(lengths))):
        x[end:] = NAN
    dq_, k_, v_, g_ = (torch.cat([times(R, x[:end].cuda()), x[end:].cuda()])
                       for x, end in ((q, sum(lengths)), (k, sum(keys)), (v, sum(keys)), (g, sum(lengths))))
    o, lse = torch.full(dq_.shape, 7.0, dtype=dtype, device="cuda"), torch.full(dq_.shape[:2], 7.0, device="cuda")
    kw = dict(cu_seqlens_k=None if past is None else cu_k.cuda(), window=window)
    gdn2.attn_fwd_varlen(dq_, k_, v_, cu.cuda(), o=o, lse=lse, **kw)
    grads = {m: torch.full(x.shape, 7.0, dtype=dtype, device="cuda") for m, x in (("dq", dq_), ("dk", k_), ("dv", v_))}
    gdn2.attn_bwd_varlen(g_, dq_, k_, v_, o, lse, cu.cuda(), grads=grads, **kw)
    torch.cuda.synchronize()
    for i in range(n):
        a, b, c, e = int(cu[i]), int(cu[i + 1]), int(cu_k[i]), int(cu_k[i + 1])
        if a < b:
            check_fwd(q[a:b], k[c:e], v[c:e], o[a:b], lse[a:b], window)
        if a < b and c < e:
            check_bwd(g[a:b], q[a:b], k[c:e], v[c:e], o[a:b], lse[a:b], dict(dq=grads["dq"][a:b], dk=grads["dk"][c:e], dv=grads["dv"][c:e]), window)
        elif c < e:
            assert not grads["dk"][c:e].any() and not grads["dv"][c:e].any()  # keys without queries
    for x, per in ((o, lengths), (lse, lengths), (grads["dq"], lengths), (grads["dk"], keys), (grads["dv"], keys)):
        end = sum(per) * R
        assert (x[end:] == 7.0).all()
        first_of(R, x[:end])


def test_packed_equals_whole():
    """Packed sequences of one length against whole ones, many of them: bit by bit."""
    B, T, H, G, d = 70, 40, 4, 2, 64
    q, k, v, g = (x.cuda() for x in case(BF16, T, T, H, G, d, 4, B))
    cu = (torch.arange(B + 1, dtype=torch.int64) * T).cuda()
    flat = [x.reshape(B * T, *x.shape[2:]) for x in (q, k, v, g)]
    o, lse = gdn2.attn_fwd(q, k, v, window=17)
    o2, lse2 = gdn2.attn_fwd_varlen(*flat[:3], cu, window=17)
    assert torch.equal(o.reshape(o2.shape), o2) and torch.equal(lse.reshape(lse2.shape), lse2)
    a, b = gdn2.attn_bwd(g, q, k, v, o, lse, window=17), gdn2.attn_bwd_varlen(flat[3], *flat[:3], o2, lse2, cu, window=17)
    assert all(torch.equal(a[n].reshape(b[n].shape), b[n]) for n in a)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_parts_of_the_keys_against_whole(dtype):
    """The same call with and without a workspace, which takes the keys in parts, between guard bytes."""
    import ctypes

    q, k, v, _ = case(dtype, 6, 3001, 4, 2, 64, 8)
    need = gdn2.attn_fwd_workspace_bytes(1, 6, 3001, 4, 2, 64, dtype=dtype)
    assert need > 0
    dev = [x.cuda() for x in (q, k, v)]
    buf = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    o, lse = gdn2.attn_fwd(*dev, workspace=buf[256:256 + need + 16])
    o2, lse2 = torch.empty_like(o), torch.empty_like(lse)
    st = gdn2._load().gdn2_attn_fwd(*[x.data_ptr() for x in (*dev, o2, lse2)], 1, 6, 3001, 4, 2, 64, 256, 128, 128, 0, 0.125,
                                    0 if dtype == F32 else 1, None, 0, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    torch.cuda.synchronize()
    assert (buf[:256] == 0x5a).all() and (buf[256 + need + 16:] == 0x5a).all()
    for x, y in ((o, lse), (o2, lse2)):
        check_fwd(q[0], k[0], v[0], x[0], y[0])


@pytest.mark.parametrize("dtype,B,T,S,H,G,d", [(BF16, 1, 700, 700, 8, 1, 64), (F32, 2, 90, 130, 6, 2, 128), (BF16, 40, 65, 65, 2, 2, 128)])
def test_gradients_keep_to_their_workspace(dtype, B, T, S, H, G, d):
    """In a caller's workspace between guard bytes, which it need not clear: the same bits."""
    q, k, v, g = (x.cuda() for x in case(dtype, T, S, H, G, d, 21, B))
    o, lse = gdn2.attn_fwd(q, k, v)
    want = gdn2.attn_bwd(g, q, k, v, o, lse)
    need = gdn2.attn_bwd_workspace_bytes(B, T, S, H, G, d, dtype=dtype)
    for fill in (0x5a, 0xff):
        buf = torch.full((need + 512,), fill, dtype=torch.uint8, device="cuda")
        got = gdn2.attn_bwd(g, q, k, v, o, lse, workspace=buf[256:256 + need + 16])
        assert all(torch.equal(want[n], got[n]) for n in want)
        assert (buf[:256] == fill).all() and (buf[256 + need + 16:] == fill).all()


def test_many_long_sequences():
    """Blocks of 256 queries: one sequence 64 times, also with values that are not finite."""
    q, k, v, _ = case(BF16, 2100, 2130, 1, 1, 128, 31)
    dev = [times(64, x.cuda()) for x in (q, k, v)]
    o, lse = first_of(64, *gdn2.attn_fwd(*dev))
    check_fwd(q[0], k[0], v[0], o[0], lse[0])
    for at, bad in ((0, NAN), (1033, INF), (2129, -INF)):
        dirty = v.clone()
        dirty[0, at, 0, 7] = bad
        o2, lse2 = first_of(64, *gdn2.attn_fwd(dev[0], dev[1], times(64, dirty.cuda())))
        assert torch.equal(lse, lse2)
        sees = torch.from_numpy(A.sees(2100, 2130, None)[:, at])
        assert torch.equal(o[0, :, 0, :7], o2[0, :, 0, :7]) and torch.equal(o[0, :, 0, 8:], o2[0, :, 0, 8:])
        assert torch.equal(o[0, ~sees, 0, 7], o2[0, ~sees, 0, 7])
        got = o2[0, sees, 0, 7].float().cpu()
        assert torch.isnan(got).all() if bad != bad else (got == bad).all()


def test_addresses_past_32_bits():
    """Tokens two million elements apart: the last ones lie past 2^32 bytes."""
    T, stride = 1100, 1 << 21
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("needs 24 GB")
    wide = torch.empty(T * stride, dtype=BF16, device="cuda")
    g = torch.Generator("cpu").manual_seed(6)
    x = torch.randn(T, 4 * 64, generator=g).to(BF16)
    rows = wide.as_strided((T, 4 * 64), (stride, 1))
    rows.copy_(x.cuda())
    q, k, v = (t[None] for t in parts(rows, 2, 1, 64))
    qc, kc, vc = (t[None] for t in parts(x, 2, 1, 64))
    o, lse = gdn2.attn_fwd(q, k, v, window=300)
    want, lw = gdn2.attn_fwd(qc.cuda(), kc.cuda(), vc.cuda(), window=300)
    assert torch.equal(o, want) and torch.equal(lse, lw)
    check_fwd(qc[0], kc[0], vc[0], o[0], lse[0], 300)
    d_o = torch.randn(o.shape, generator=g).to(BF16).cuda()
    a, b = gdn2.attn_bwd(d_o, q, k, v, o, lse, window=300), gdn2.attn_bwd(d_o, qc.cuda(), kc.cuda(), vc.cuda(), o, lse, window=300)
    assert all(torch.equal(a[n], b[n]) for n in a)


# ---- values that are not finite -------------------------------------------------------------

@MANY
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
@pytest.mark.parametrize("T,window,at", [(200, None, 90), (200, 50, 90), (70, 7, 33), (300, 129, 128), (64, None, 0)])
def test_bad_values_reach_no_query_that_does_not_see_them(dtype, bad, T, window, at, many):
    H, G, d = 2, 1, 64
    q, k, v, g = case(dtype, T, T, H, G, d, T + at)
    seen = A.sees(T, T, window)[:, at]  # the queries that see token `at`
    clean = [x.cuda() for x in (q, k, v)]
    o, lse = fwd(many, *clean, window=window)
    dirty_v = v.clone()
    dirty_v[0, at, 0, 5] = bad
    o2, lse2 = fwd(many, clean[0], clean[1], dirty_v.cuda(), window=window)
    assert torch.equal(lse, lse2)
    hit = torch.zeros(T, d, dtype=torch.bool)
    hit[:, 5] = torch.from_numpy(seen)
    same = ~hit[None, :, None].expand(1, T, H, d).cuda()
    assert torch.equal(o[same], o2[same])
    want = torch.full_like(o2[~same], bad)
    assert torch.equal(torch.nan_to_num(o2[~same], 1.0, 2.0, 3.0), torch.nan_to_num(want, 1.0, 2.0, 3.0))
    dirty_k = k.clone()
    dirty_k[0, at] = bad
    o3, lse3 = fwd(many, clean[0], dirty_k.cuda(), clean[2], window=window)
    blind = torch.from_numpy(~seen).cuda()
    assert torch.equal(o[:, blind], o3[:, blind]) and torch.equal(lse[:, blind], lse3[:, blind])
    # gradients: an upstream gradient, a key and a value of one token
    grads = bwd(many, g.cuda(), *clean, o, lse, window=window)
    dirty_g = g.clone()
    dirty_g[0, at, :, 7] = bad
    bad_g = bwd(many, dirty_g.cuda(), *clean, o, lse, window=window)
    others = torch.arange(T, device="cuda") != at
    assert torch.equal(grads["dq"][:, others], bad_g["dq"][:, others])
    unseen = torch.from_numpy(~A.sees(T, T, window)[at]).cuda()  # keys that query `at` does not see
    for n in ("dk", "dv"):
        assert torch.equal(grads[n][:, unseen], bad_g[n][:, unseen]), n
    assert not torch.isfinite(bad_g["dv"][:, ~unseen][..., 7]).any()
    assert torch.equal(grads["dv"][..., :7], bad_g["dv"][..., :7])
    ok, lk = fwd(many, clean[0], dirty_k.cuda(), clean[2], window=window)
    bad_k = bwd(many, g.cuda(), clean[0], dirty_k.cuda(), clean[2], ok, lk, window=window)
    assert torch.equal(grads["dq"][:, blind], bad_k["dq"][:, blind])
    far = torch.from_numpy(~(A.sees(T, T, window)[seen].any(0))).cuda()  # keys that no query of those sees
    for n in ("dk", "dv"):
        assert torch.equal(grads[n][:, far], bad_k[n][:, far]), n
    dirty_q = q.clone()
    dirty_q[0, at] = bad
    oq, lq = fwd(many, dirty_q.cuda(), *clean[1:], window=window)
    assert torch.equal(o[:, others], oq[:, others])
    bad_q = bwd(many, g.cuda(), dirty_q.cuda(), *clean[1:], oq, lq, window=window)
    assert torch.equal(grads["dq"][:, others], bad_q["dq"][:, others])
    for n in ("dk", "dv"):
        assert torch.equal(grads[n][:, unseen], bad_q[n][:, unseen]), n


# ---- steps ----------------------------------------------------------------------------------

STEPS = [  # dtype, positions, C, H, G, d, window
    (BF16, [0, 1, 5], 8, 2, 1, 64, None), (BF16, [7, 8, 20, 31], 8, 4, 2, 128, None), (BF16, [3, 100, 63, 64, 200, -1], 64, 8, 2, 128, 33),
    (BF16, [500, 1023, 1024, 5000, 0], 1024, 16, 2, 128, None), (BF16, [40], 2048, 6, 2, 64, 16), (BF16, [2999, -7, 31], 3000, 1, 1, 64, 2000),
    (BF16, [90, 33], 100, 40, 1, 64, None), (BF16, [90, 33], 100, 33, 1, 128, 64),
    (F32, [0, 31, 32, 33], 40, 2, 1, 64, None), (F32, [700, 6], 600, 6, 3, 128, None), (F32, [129], 128, 4, 1, 128, 100),
]


@pytest.mark.parametrize("dtype,places,C,H,G,d,window", STEPS)
def test_step_matches_oracle(dtype, places, C, H, G, d, window):
    say("case: step %s positions %s C%d H%d G%d d%d window %s" % (dtype, places, C, H, G, d, window))
    n = len(places)
    g = torch.Generator("cpu").manual_seed(C + H)
    r = lambda *s: torch.randn(s, generator=g).to(dtype)
    qkv, kc, vc = r(n, (H + 2 * G) * d), r(n, C, G, d), r(n, C, G, d)
    for i, p in enumerate(places):  # slots that hold no token yet may be anything
        kc[i, max(p, 0) if p < C else C:] = NAN
        vc[i, max(p, 0) if p < C else C:] = INF
    q, k, v = parts(qkv.cuda(), H, G, d)
    k_cache, v_cache = kc.cuda(), vc.cuda()
    o = gdn2.attn_step(q, k, v, k_cache, v_cache, torch.tensor(places, dtype=torch.int64, device="cuda"), window=window)
    torch.cuda.synchronize()
    q, k, v = parts(qkv, H, G, d)
    for i, p in enumerate(places):
        wk, wv = kc[i].clone(), vc[i].clone()
        if p >= 0:
            wk[p % C], wv[p % C] = k[i], v[i]
        assert torch.equal(torch.nan_to_num(wk, 9.0), torch.nan_to_num(k_cache[i].cpu(), 9.0)) and torch.equal(wv, v_cache[i].cpu())
        if p < 0:
            assert not o[i].any()
            continue
        tokens = torch.arange(max(0, p + 1 - min(C, window or C)), p + 1) % C
        check_fwd(q[i:i + 1], wk[tokens], wv[tokens], o[i:i + 1], None)


def test_step_past_32_bits():
    """A cache of more than 2^32 bytes a sequence, its last slots and the way round."""
    C, G, d = (1 << 24) + 40, 2, 64
    if torch.cuda.mem_get_info()[0] < 40 << 30:
        pytest.skip("needs 40 GB")
    kc, vc = torch.zeros(2, C, G, d, dtype=BF16, device="cuda"), torch.zeros(2, C, G, d, dtype=BF16, device="cuda")
    g = torch.Generator("cpu").manual_seed(1)
    places = [C - 2, C + 20]
    fill = torch.randn(2, 2, 300, G, d, generator=g).to(BF16)
    for i, p in enumerate(places):
        at = (torch.arange(p - 300, p) % C).cuda()
        kc[i, at], vc[i, at] = fill[i, 0].cuda(), fill[i, 1].cuda()
    q, k, v = (torch.randn(2, n, d, generator=g).to(BF16) for n in (4, G, G))
    o = gdn2.attn_step(q.cuda(), k.cuda(), v.cuda(), kc, vc, torch.tensor(places, device="cuda"), window=290)
    for i in range(2):
        check_fwd(q[i:i + 1], torch.cat((fill[i, 0, -289:], k[i:i + 1])), torch.cat((fill[i, 1, -289:], v[i:i + 1])), o[i:i + 1], None)
        assert torch.equal(kc[i, places[i] % C].cpu(), k[i]) and torch.equal(vc[i, places[i] % C].cpu(), v[i])


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_step_in_parts_against_whole(dtype):
    import ctypes

    g = torch.Generator("cuda").manual_seed(2)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(dtype)
    q, k, v, kc, vc = r(2, 4, 64), r(2, 2, 64), r(2, 2, 64), r(2, 5000, 2, 64), r(2, 5000, 2, 64)
    places = torch.tensor([4321, 9999], device="cuda")
    need = gdn2.attn_step_workspace_bytes(2, 4, 2, 64, 5000, dtype=dtype)
    assert need > 0
    k2, v2 = kc.clone(), vc.clone()
    buf = torch.full((need + 512,), 0x5a, dtype=torch.uint8, device="cuda")
    o = gdn2.attn_step(q, k, v, kc, vc, places, workspace=buf[256:256 + need + 16])
    o2 = torch.empty_like(o)
    st = gdn2._load().gdn2_attn_step(*[x.data_ptr() for x in (q, k, v, k2, v2, places, o2)], 2, 4, 2, 64, 5000, 256, 128, 128, 0, 0.125,
                                     0 if dtype == F32 else 1, None, 0, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream))
    assert st == 0
    torch.cuda.synchronize()
    assert (buf[:256] == 0x5a).all() and (buf[256 + need + 16:] == 0x5a).all()
    assert torch.equal(kc, k2) and torch.equal(vc, v2)
    for i, p in enumerate(places.tolist()):
        tokens = torch.arange(max(0, p + 1 - 5000), p + 1, device="cuda") % 5000
        for x in (o, o2):
            check_fwd(q[i:i + 1].cpu(), kc[i, tokens].cpu(), vc[i, tokens].cpu(), x[i:i + 1], None)


# ---- rotary ---------------------------------------------------------------------------------

ROTARY = [  # dtype, lead, H, G, d, rot, interleaved, far
    (BF16, (2, 7), 4, 2, 64, 64, False, 0), (BF16, (2, 7), 4, 2, 64, 64, True, 0), (BF16, (1, 1), 16, 2, 128, 64, False, 1 << 20),
    (BF16, (300,), 3, 1, 128, 32, False, 1 << 30), (F32, (3, 40), 2, 2, 64, 32, True, 1 << 20), (F32, (1, 1300), 2, 1, 128, 128, False, 0),
    (F32, (9,), 1, 0, 6, 4, False, 100), (BF16, (9,), 3, 1, 10, 6, True, 100), (BF16, (5,), 2, 1, 64, 12, False, 7), (F32, (4,), 2, 1, 512, 512, False, 3),
    (BF16, (2500,), 40, 2, 128, 128, True, 0), (BF16, (1100,), 2, 1, 128, 126, False, 0),
    (BF16, (33,), 3, 1, 96, 48, False, 9), (F32, (21,), 2, 2, 96, 48, True, 9), (BF16, (40,), 5, 1, 8, 8, True, 50), (F32, (3000,), 1, 0, 16, 8, False, 0),
]


def rotary_bar(x, freq, inter, scale=1.0):
    n = freq.shape[0]
    a = np.abs(f64(x))
    pair = a.copy()
    first, second = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if inter else (slice(0, n), slice(n, 2 * n))
    pair[..., first] = pair[..., second] = a[..., first] + a[..., second]
    pair[..., 2 * n:] = 0
    return 12 * U * scale * pair


@pytest.mark.parametrize("dtype,lead,H,G,d,rot,inter,far", ROTARY)
def test_rotary_matches_oracle(dtype, lead, H, G, d, rot, inter, far):
    say("case: rotary %s %s H%d G%d d%d rot %d interleaved %s far %d" % (dtype, lead, H, G, d, rot, inter, far))
    g = torch.Generator("cpu").manual_seed(d + rot)
    q, k = torch.randn(*lead, H, d, generator=g).to(dtype), torch.randn(*lead, max(G, 1), d, generator=g).to(dtype)
    freq = gdn2.rotary_frequencies(rot, 1000.0)
    places = torch.randint(-5, far, lead, generator=g) if far else None
    dev = None if places is None else places.cuda()
    at = np.broadcast_to(np.arange(lead[-1]), lead) if places is None else places.numpy()
    qo, ko = gdn2.rotary(q.cuda(), k.cuda() if G else None, freq.cuda(), dev, interleaved=inter, scale=1.25)
    for name, x, y in (("q", q, qo), ("k", k, ko))[:2 if G else 1]:
        ref = A.rotary(x, freq, at, inter, scale=1.25)
        within(name, y, ref, rotary_bar(x, freq, inter, 1.25) + half_step(dtype) * np.abs(ref))
        assert torch.equal(y[..., rot:].cpu(), x[..., rot:])
        back = gdn2.rotary(x.cuda(), None, freq.cuda(), dev, interleaved=inter, inverse=True)[0]
        ref = A.rotary(x, freq, at, inter, inverse=True)
        within(name + " back", back, ref, rotary_bar(x, freq, inter) + half_step(dtype) * np.abs(ref))
    if G == 0:
        assert ko is None


@pytest.mark.parametrize("dtype,extra", [(BF16, 0), (BF16, 8), (F32, 3)])
def test_rotary_in_place_on_parts_of_one_tensor(dtype, extra):
    H, G, d, rot = 4, 2, 64, 32
    g = torch.Generator("cuda").manual_seed(3)
    qkv = torch.randn(2, 50, (H + 2 * G) * d + extra, generator=g, device="cuda").to(dtype)
    before = qkv.clone()
    q, k, v = parts(qkv[..., :(H + 2 * G) * d], H, G, d)
    freq = gdn2.rotary_frequencies(rot, device="cuda")
    want = gdn2.rotary(q, k, freq)
    got = gdn2.rotary(q, k, freq, q_out=q, k_out=k)
    assert got[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(qkv[..., (H + G) * d:], before[..., (H + G) * d:])  # values and what lies between tokens
    # into another wide tensor, q alone in place
    other = torch.zeros_like(before)
    qb, kb, _ = parts(before[..., :(H + 2 * G) * d], H, G, d)
    _, ko, _ = parts(other[..., :(H + 2 * G) * d], H, G, d)
    gdn2.rotary(qb, kb, freq, q_out=qb, k_out=ko)
    assert torch.equal(qb, want[0]) and torch.equal(ko, want[1])
    for bad in (dict(q_out=k.expand_as(k)), dict(k_out=q[..., :G, :]), dict(q_out=qkv[..., 8:8 + H * d].unflatten(-1, (H, d)))):
        with pytest.raises((gdn2.Gdn2Error, ValueError)):
            gdn2.rotary(q, k, freq, **bad)


# ---- norm -----------------------------------------------------------------------------------

NORMS = [(1, 1), (3, 7), (5, 64), (130, 127), (9, 300), (33, 512), (7, 1000), (4, 1540), (6, 2048), (3, 4096), (5, 8192), (2, 9001), (2, 16384), (9000, 70),
         (600, 1024), (300, 4097)]


@pytest.mark.parametrize("rows,width", NORMS)
@pytest.mark.parametrize("dtype,rdtype", [(BF16, None), (BF16, BF16), (BF16, F32), (F32, F32)])
def test_rms_norm_matches_oracle(dtype, rdtype, rows, width):
    say("case: norm %s residual %s %d x %d" % (dtype, rdtype, rows, width))
    g = torch.Generator("cpu").manual_seed(rows + width)
    x, gamma = torch.randn(rows, width, generator=g).to(dtype), torch.randn(width, generator=g)
    res = None if rdtype is None else (3 * torch.randn(rows, width, generator=g)).to(rdtype)
    if rows > 1:
        x[1] = 0
        if res is not None:
            res[1] = 0
    dev = [None if t is None else t.cuda() for t in (x, gamma, res)]
    ry, rh, rr = A.rms_norm(x, gamma, 1e-5, res)
    sums = np.abs(f64(x)) + (0 if res is None else np.abs(f64(res)))
    y, h, rstd = gdn2.rms_norm(dev[0], dev[1], 1e-5, residual=dev[2])
    # h is one rounded sum: against terms that cancel it is off by a half step of the result, no more
    gr = np.abs(f64(gamma)) * rr[:, None]
    loss = np.sqrt((sums ** 2).mean(-1)) * rr  # the sums' roundings in the mean of squares
    ty = (52 * U + U * loss[:, None] + 4 * U) * np.abs(ry) + U * gr * np.abs(rh)
    within("y", y, ry, ty + half_step(dtype) * np.abs(ry))
    within("rstd", rstd, rr, rr * (52 + loss) * U)
    if res is None:
        assert h is None
    else:
        assert torch.equal(h.cpu(), (x.float() + res.float()).to(rdtype))
    y8, scales, h8, rstd8 = gdn2.rms_norm_fp8(dev[0], dev[1], 1e-5, residual=dev[2])
    assert torch.equal(rstd8, rstd) and (res is None or torch.equal(h8, h)) and y8.dtype == torch.float8_e4m3fn
    top = np.abs(ry).max(-1)
    rs = np.where(top > 0, top / A.E4M3_MAX, 1.0)
    within("scales", scales, rs, 64 * U * rs * (1 + loss))
    sc = f64(scales)[:, None]
    within("8 bits", y8.float() * scales[:, None], ry, np.maximum(2.0 ** -4 * np.abs(ry), 2.0 ** -10 * sc) * (1 + 2.0 ** -18) + ty)
    only = gdn2.rms_norm(dev[0], dev[1], 1e-5, residual=dev[2], stats=False)
    assert only[2] is None and torch.equal(only[0], y)


@pytest.mark.parametrize("rows,width", NORMS)
@pytest.mark.parametrize("dtype,hdtype,stream", [(BF16, BF16, True), (BF16, F32, True), (F32, F32, False)])
def test_rms_norm_gradients_match_oracle(dtype, hdtype, stream, rows, width):
    say("case: norm gradients %s h %s %d x %d" % (dtype, hdtype, rows, width))
    g = torch.Generator("cpu").manual_seed(rows * 3 + width)
    h, gamma = (2 * torch.randn(rows, width, generator=g)).to(hdtype), torch.randn(width, generator=g)
    dy = torch.randn(rows, width, generator=g).to(dtype)
    dh = torch.randn(rows, width, generator=g).to(hdtype) if stream else None
    rstd = torch.from_numpy(A.rms_norm(h, gamma, 1e-5)[2]).float()
    dx, dg = A.rms_norm_bwd(dy, h, gamma, rstd, dh)
    dev = [None if t is None else t.cuda() for t in (dy, h, gamma, rstd, dh)]
    out = gdn2.rms_norm_bwd(*dev[:4], dh=dev[4])
    u, v = np.abs(f64(h)) * f64(rstd)[:, None], np.abs(f64(dy) * f64(gamma))
    size = f64(rstd)[:, None] * (v + u * (u * v).mean(-1, keepdims=True)) + (0 if dh is None else np.abs(f64(dh)))
    within("dx", out["dx"], dx, 110 * U * size + half_step(hdtype) * np.abs(dx))
    within("dgamma", out["dgamma"], dg, 600 * U * (np.abs(f64(dy)) * u).sum(0))
    if stream:  # in the place of the stream's gradient
        again = gdn2.rms_norm_bwd(*dev[:4], dh=dev[4], grads=dict(dx=dev[4]))
        assert again["dx"] is dev[4] and torch.equal(again["dx"], out["dx"]) and torch.equal(again["dgamma"], out["dgamma"])


@pytest.mark.parametrize("size", [2.0 ** -109, 2.0 ** -112, 2.0 ** -120, 2.0 ** -126])
def test_rms_norm_fp8_of_tiny_rows(size):
    """Rows so small that 448 over the largest value leaves fp32: zeros stay zeros, the others within a half step."""
    x = torch.ones(3, 96)
    x[1, ::2], x[2, 5:] = 0, 0
    gamma = torch.full((96,), size)
    y, scales, _, _ = gdn2.rms_norm_fp8(x.cuda(), gamma.cuda(), 1e-6)
    ref = A.rms_norm(x, gamma, 1e-6)[0]
    s, got = f64(scales)[:, None], f64(y.float()) * f64(scales)[:, None]
    assert np.isfinite(got).all() and (s > 0).all()
    bar = np.maximum(2.0 ** -4 * np.abs(ref), 2.0 ** -10 * s) + 64 * U * np.abs(ref)
    assert (np.abs(got - ref) <= bar).all() and (got[ref == 0] == 0).all()


def test_norm_of_no_rows_and_in_place():
    gamma = torch.rand(64, device="cuda")
    y, h, rstd = gdn2.rms_norm(torch.empty(0, 64, dtype=BF16, device="cuda"), gamma, residual=torch.empty(0, 64, device="cuda"))
    assert y.shape == (0, 64) and h.dtype == F32 and rstd.shape == (0,)
    e = torch.empty(0, 64, device="cuda")
    assert not gdn2.rms_norm_bwd(e, e, gamma, torch.empty(0, device="cuda"))["dgamma"].any()
    x, res = torch.randn(40, 64, device="cuda").to(BF16), torch.randn(40, 64, device="cuda")
    want = gdn2.rms_norm(x, gamma, residual=res)
    got = gdn2.rms_norm(x, gamma, residual=res, h=res)
    assert got[1] is res and torch.equal(res, want[1]) and torch.equal(got[0], want[0])


# ---- together -------------------------------------------------------------------------------

def layer(x, res, p, H, G, d, freq, positions, cu, window):
    """The attention half of a layer on packed tokens; returns its output, the stream, and what was kept."""
    y, h, rstd = gdn2.rms_norm(x, p["gamma"], residual=res)
    q, k, v = parts(y @ p["qkv"], H, G, d)
    gdn2.rotary(q, k, freq, positions, q_out=q, k_out=k)
    o, lse = gdn2.attn_fwd_varlen(q, k, v, cu, window=window)
    return o.flatten(-2) @ p["out"], h, (y, h, rstd, q, k, v, o, lse)


def setup_layer(dtype, H, G, d, width):
    g = torch.Generator("cpu").manual_seed(21)
    r = lambda *s: torch.randn(s, generator=g)
    return {"gamma": (1 + 0.1 * r(width)).cuda(), "qkv": (r(width, (H + 2 * G) * d) * width ** -0.5).to(dtype).cuda(),
            "out": (r(H * d, width) * (H * d) ** -0.5).to(dtype).cuda()}


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_a_layer_from_prompts_to_tokens(dtype):
    """Norm, projections, rotary, attention over packed prompts, then single tokens over caches of the
    window, against the whole sequences at once."""
    H, G, d, width, window, C = 4, 2, 64, 96, 20, 32
    lengths, more = [37, 5, 61], 9
    p = setup_layer(dtype, H, G, d, width)
    freq = gdn2.rotary_frequencies(d // 2, device="cuda")
    g = torch.Generator("cpu").manual_seed(4)
    full = [torch.randn(2, n + more, width, generator=g).to(dtype).cuda() for n in lengths]
    whole = []
    for f in full:
        n = f.shape[1]
        out, h, _ = layer(f[0], f[1], p, H, G, d, freq, torch.arange(n, device="cuda"), torch.tensor([0, n], device="cuda"), window)
        whole.append((out, h))
    cu = offsets(lengths).cuda()
    x, res = (torch.cat([f[i, :n] for f, n in zip(full, lengths)]) for i in (0, 1))
    places = torch.cat([torch.arange(n) for n in lengths]).cuda()
    out, h, kept = layer(x, res, p, H, G, d, freq, places, cu, window)
    tol = 2.0 ** -5 if dtype == BF16 else 2.0 ** -15  # a few roundings of sums of terms of size one
    for i, n in enumerate(lengths):
        a = int(cu[i])
        assert (out[a:a + n].float() - whole[i][0][:n].float()).abs().max() <= tol
        assert torch.equal(h[a:a + n], whole[i][1][:n])
    k_cache = torch.zeros(len(lengths), C, G, d, dtype=dtype, device="cuda")
    v_cache = torch.zeros_like(k_cache)
    for i, n in enumerate(lengths):  # the prompts' last tokens into their slots
        a, tokens = int(cu[i]), torch.arange(max(0, n - C), n, device="cuda")
        k_cache[i, tokens % C], v_cache[i, tokens % C] = kept[4][a + tokens], kept[5][a + tokens]
    positions = torch.tensor(lengths, device="cuda")
    for j in range(more):
        x, res = (torch.stack([f[i, n + j] for f, n in zip(full, lengths)]) for i in (0, 1))
        y, h, _ = gdn2.rms_norm(x, p["gamma"], residual=res)
        q, k, v = parts(y @ p["qkv"], H, G, d)
        gdn2.rotary(q, k, freq, positions, q_out=q, k_out=k)
        o = gdn2.attn_step(q, k, v, k_cache, v_cache, positions, window=window)
        out = o.flatten(-2) @ p["out"]
        for i, n in enumerate(lengths):
            assert (out[i].float() - whole[i][0][n + j].float()).abs().max() <= tol, (j, i)
        positions += 1


def test_a_layers_gradients_against_differences():
    """The backward pass of the same chain in fp32, from the calls' gradients, against slopes in 64 bits
    of the oracle's chain."""
    H, G, d, width, window = 2, 1, 64, 48, 11
    p = setup_layer(F32, H, G, d, width)
    freq = gdn2.rotary_frequencies(d, device="cuda")
    n = 30
    g = torch.Generator("cpu").manual_seed(9)
    x, res, w, wh = (torch.randn(n, width, generator=g) for _ in range(4))
    places, cu = torch.arange(n, device="cuda"), torch.tensor([0, n], device="cuda")
    _, _, (y, h, rstd, q, k, v, o, lse) = layer(x.cuda(), res.cuda(), p, H, G, d, freq, places, cu, window)
    d_o = (w.cuda() @ p["out"].T).unflatten(-1, (H, d))
    grads = gdn2.attn_bwd_varlen(d_o, q, k, v, o, lse, cu, window=window)
    dq, dk = gdn2.rotary(grads["dq"], grads["dk"], freq, places, inverse=True)
    dy = torch.cat([t.flatten(-2) for t in (dq, dk, grads["dv"])], -1) @ p["qkv"].T
    out = gdn2.rms_norm_bwd(dy, h, p["gamma"], rstd, dh=wh.cuda())

    def loss(x, res, gamma):
        y, h, _ = A.rms_norm(x, gamma, 1e-6, res)
        q, k, v = (t.numpy() for t in parts(torch.from_numpy(y) @ p["qkv"].cpu().double(), H, G, d))
        f, at = freq.cpu(), np.arange(n)
        o, _ = A.attention(A.rotary(q, f, at), A.rotary(k, f, at), v, window)
        return ((o.reshape(n, -1) @ f64(p["out"])) * f64(w)).sum() + (h * f64(wh)).sum()

    args = [f64(x), f64(res), f64(p["gamma"])]
    r = np.random.default_rng(1)
    for at, grad in ((0, out["dx"]), (1, out["dx"]), (2, out["dgamma"])):
        way = r.normal(size=args[at].shape)
        up, down = (loss(*[a + s * 1e-5 * way if i == at else a for i, a in enumerate(args)]) for s in (1, -1))
        want = (f64(grad) * way).sum()
        size = (np.abs(f64(grad)) * np.abs(way)).sum()
        assert abs((up - down) / 2e-5 - want) <= 1e-5 * size + 1e-7, (at, (up - down) / 2e-5, want)


def test_streams_and_replayed_graphs():
    """Captured calls (workspaces and all) replayed on new values between eager work, on another stream."""
    g = torch.Generator("cuda").manual_seed(5)
    r = lambda *s: torch.randn(s, generator=g, device="cuda").to(BF16)
    q, k, v, d_o = r(1, 40, 4, 64), r(1, 2000, 2, 64), r(1, 2000, 2, 64), r(1, 40, 4, 64)
    sq, sk, sv, kc, vc = r(3, 4, 64), r(3, 2, 64), r(3, 2, 64), r(3, 3000, 2, 64), r(3, 3000, 2, 64)
    places = torch.tensor([2999, 17, 4000], device="cuda")
    x, res, gamma, dy = r(900, 640), torch.randn(900, 640, generator=g, device="cuda"), torch.rand(640, device="cuda"), r(900, 640)
    freq = gdn2.rotary_frequencies(64, device="cuda")

    def run():
        a, b = gdn2.rotary(q, k[:, :40], freq)
        o, lse = gdn2.attn_fwd(q, k, v)
        grads = gdn2.attn_bwd(d_o, q, k, v, o, lse)
        s = gdn2.attn_step(sq, sk, sv, kc, vc, places)
        y, h, rstd = gdn2.rms_norm(x, gamma, residual=res)
        y8 = gdn2.rms_norm_fp8(x, gamma, residual=res)
        back = gdn2.rms_norm_bwd(dy, h, gamma, rstd, dh=h)
        return [a, b, o, lse, *grads.values(), s, kc, vc, y, h, rstd, y8[0].view(torch.uint8), y8[1], back["dx"], back["dgamma"]]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            outs = run()
    torch.cuda.current_stream().wait_stream(side)
    for turn in range(4):
        for t in (q, k, v, d_o, sq, sk, sv, x, dy):
            t.copy_(r(*t.shape))
        torch.cuda.synchronize()
        before = [kc.clone(), vc.clone()]
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in outs]
        kc.copy_(before[0])
        vc.copy_(before[1])
        want = run()  # eager, on the current stream
        torch.cuda.synchronize()
        for i, (a, b) in enumerate(zip(got, want)):
            assert torch.equal(a, b), (turn, i)


def test_outputs_are_written_in_full_and_nothing_else():
    """Outputs between guard rows, filled with NaN before the call."""
    q, k, v, g = (x.cuda() for x in case(BF16, 130, 130, 2, 1, 128, 3))

    def guarded(shape, dtype):
        n = math.prod(shape)
        buf = torch.full((n + 256,), NAN, dtype=dtype, device="cuda")
        return buf, buf[128:128 + n].view(shape)

    bufs = {n: guarded(s, t) for n, s, t in (("o", q.shape, BF16), ("lse", (1, 130, 2), F32), ("dq", q.shape, BF16), ("dk", k.shape, BF16),
                                             ("dv", v.shape, BF16))}
    gdn2.attn_fwd(q, k, v, o=bufs["o"][1], lse=bufs["lse"][1])
    gdn2.attn_bwd(g, q, k, v, bufs["o"][1], bufs["lse"][1], grads={n: bufs[n][1] for n in ("dq", "dk", "dv")})
    torch.cuda.synchronize()
    for n, (buf, t) in bufs.items():
        assert torch.isfinite(t).all(), n
        assert torch.isnan(buf[:128]).all() and torch.isnan(buf[-128:]).all(), n
