"""GPU parity of the state space block (scan, short convolution, layer norm) with its fp64 oracle.

Bars, element by element, from the arithmetic (u = 2^-24, the half step of fp32; a bf16 rounding
is off by at most 2^-8 of the value):

* scan, fp32: a term of y or S is a product of a few factors, its decays exp of an argument that
  is rounded once (below 88 in size, or the term is gone: 88 u), and passes at most 64 additions
  in its chunk's sum, 128 over the state's rows and three roundings a chunk that it is carried
  through, so |y - ref| <= (320 + 4 chunks) u Y with Y the same sum over absolute values.
* scan, bf16: inputs enter as they are.  The pair weights of a chunk are rounded to bf16 once, a
  state where it is read for y once, and y on the store, so 2^-8 (1 + 2^-7) of Y's terms but D x,
  and 2^-8 |y|, come on top.  Final states are held to the fp32 bound.
* convolution: five products and sums (8 u U, U the sum of absolute values, and SiLU's slope is
  below 1.1), then a sigmoid whose exponential's argument is rounded (8 + 4 |u| roundings of |y|);
  the store's 2^-8 |y| in bf16.  States are copies: equal bits.
* norm: sums over a row pass at most 96 roundings (64 elements of a lane and the tree), so the
  mean is off by 100 u mean|x|, rstd by 120 u of itself, and y, dx by those carried through;
  sums over rows at most 600 roundings."""
import numpy as np
import pytest
import torch

import gated_delta_rule_gdn2_amd as gdn2
from oracle import block as O
from tests.parity_util import say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")
    gdn2._load()


def f64(t):
    return t.detach().cpu().double().numpy()


def within(name, got, ref, tol):
    got = f64(got)
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    assert np.isfinite(got).all(), name
    worst = float((np.abs(got - ref) / (tol + 1e-30)).max()) if got.size else 0.0
    say("  %-12s worst %.3f of its bar" % (name, worst))
    assert worst <= 1.0, (name, worst)


# ---- scan -----------------------------------------------------------------------------------

def scan_case(dtype, lead, H, G, dk, dv, seed, states=None, strong=False):
    g = torch.Generator("cpu").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    k = dict(x=r(*lead, H, dv).to(dtype), dt=(0.5 * r(*lead, H)).to(dtype), B=r(*lead, G, dk).to(dtype),
             C=r(*lead, G, dk).to(dtype), A=-(torch.rand(H, generator=g) * 15 + 1) * (8 if strong else 1), D=r(H),
             dt_bias=r(H) - (0 if strong else 4))
    k["s0"] = None if states is None else 0.5 * r(states, H, dk, dv)
    return k


def dev(k):
    return {n: None if v is None else v.cuda() for n, v in k.items()}


def oracle_scan(k, softplus=True):
    """(y, S) and the sums of absolute values (Y without D x, S)."""
    args = [k[n] for n in ("x", "dt", "B", "C", "A")]
    y, s = O.ssm(*args, k["D"], k["dt_bias"], k["s0"], softplus)
    ab = lambda t: None if t is None else np.abs(f64(t))
    ya, sa = O.ssm(ab(k["x"]), k["dt"], ab(k["B"]), ab(k["C"]), k["A"], None, k["dt_bias"], ab(k["s0"]), softplus)
    return y, s, ya, sa


def check_scan(k, y, s, ref, chunks):
    yr, sr, ya, sa = ref
    n = (320 + 4 * chunks) * U
    dx = 0 if k["D"] is None else np.abs(f64(k["D"])[:, None] * f64(k["x"]).reshape(yr.shape))
    tol = n * (ya + dx)
    if y.dtype == BF16:
        tol = tol + 2.0 ** -8 * (1 + 2.0 ** -7) * ya + 2.0 ** -8 * np.abs(yr)
    within("y", y, yr, tol)
    if s is not None:
        within("state", s, sr, n * sa)


SCANS = [  # dtype, B, T, H, G, dk, dv, states, strong
    (BF16, 1, 1, 1, 1, 64, 64, False, False),
    (BF16, 2, 2, 2, 1, 128, 64, True, False),
    (BF16, 3, 63, 4, 2, 64, 128, True, False),
    (BF16, 1, 64, 2, 2, 128, 128, False, True),
    (BF16, 2, 65, 6, 3, 128, 128, True, False),
    (BF16, 1, 333, 3, 1, 128, 64, True, True),
    (BF16, 1, 1000, 2, 1, 64, 64, False, False),
    (BF16, 1, 4300, 2, 2, 128, 128, True, False),
    (BF16, 1, 2111, 1, 1, 64, 128, True, True),
    (F32, 1, 1, 2, 1, 64, 64, True, False),
    (F32, 2, 65, 4, 2, 128, 64, True, False),
    (F32, 1, 200, 2, 2, 128, 128, False, True),
    (F32, 2, 333, 3, 3, 64, 128, True, False),
    (F32, 1, 2500, 2, 1, 64, 64, True, False),
    # heads of 128 columns in one workgroup each (the few heads above are in halves), whole and cut
    (BF16, 9, 70, 16, 2, 128, 128, True, False),
    (BF16, 3, 1300, 16, 1, 64, 128, True, False),
    (F32, 9, 70, 16, 1, 64, 128, True, False),
    (F32, 2, 450, 18, 2, 64, 128, True, False),
]


@pytest.mark.parametrize("dtype,B,T,H,G,dk,dv,states,strong", SCANS)
def test_scan_matches_oracle(dtype, B, T, H, G, dk, dv, states, strong):
    say("case: scan %s B%d T%d H%d G%d dk%d dv%d" % (dtype, B, T, H, G, dk, dv))
    k = scan_case(dtype, (B, T), H, G, dk, dv, 11 * T + H, B if states else None, strong)
    d = dev(k)
    y, s = gdn2.ssm_fwd(d["x"], d["dt"], d["B"], d["C"], d["A"], d["D"], d["dt_bias"], d["s0"])
    torch.cuda.synchronize()
    check_scan(k, y, s, oracle_scan(k), (T + 63) // 64)
    again, s2 = gdn2.ssm_fwd(d["x"], d["dt"], d["B"], d["C"], d["A"], d["D"], d["dt_bias"], d["s0"])
    assert torch.equal(y, again) and torch.equal(s, s2)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_without_the_optional_inputs(dtype):
    k = scan_case(dtype, (2, 70), 2, 1, 64, 64, 5)
    k.update(D=None, dt_bias=None, dt=k["dt"].abs())
    d = dev(k)
    y, s = gdn2.ssm_fwd(d["x"], d["dt"], d["B"], d["C"], d["A"], softplus=False)
    check_scan(k, y, s, oracle_scan(k, softplus=False), 2)
    y2, none = gdn2.ssm_fwd(d["x"], d["dt"], d["B"], d["C"], d["A"], softplus=False, output_final_state=False)
    assert none is None and torch.equal(y, y2)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_scan_after_tokens_that_clear_the_state(dtype):
    """A few tokens whose decay is e^-1e7 (documents joined in one sequence are set apart so): what
    follows them in the same chunk keeps its own decays, of a tenth a token."""
    k = scan_case(dtype, (1, 150), 2, 1, 64, 64, 23, 1)
    k.update(A=torch.full((2,), -1e5), dt_bias=None, dt=torch.full((1, 150, 2), 1e-6).to(dtype))
    for t in (5, 6, 70, 149):
        k["dt"][:, t] = 100.0
    k["x"] = (k["x"] * 1e3).to(dtype)
    d = dev(k)
    y, s = gdn2.ssm_fwd(d["x"], d["dt"], d["B"], d["C"], d["A"], d["D"], None, d["s0"], softplus=False)
    check_scan(k, y, s, oracle_scan(k, softplus=False), 3)


@pytest.mark.parametrize("dtype,T", [(BF16, 130), (F32, 130), (BF16, 2200)])
def test_scan_reads_parts_of_one_tensor(dtype, T):
    """x, B, C and dt as parts of wider tensors give the bits of their copies; caller outputs are
    written whole; the state may be updated in place."""
    B, H, G, dk, dv = 2, 2, 1, 64, 128
    k = scan_case(dtype, (B, T), H, G, dk, dv, 6, B)
    wide = torch.cat([k["x"].flatten(2), k["B"].flatten(2), k["C"].flatten(2)], -1).cuda()
    x, b, c = wide.split([H * dv, G * dk, G * dk], -1)
    x, b, c = x.unflatten(-1, (H, dv)), b.unflatten(-1, (G, dk)), c.unflatten(-1, (G, dk))
    dt = torch.cat([k["dt"], k["dt"]], -1).cuda()[..., H:]
    d = dev(k)
    ref = gdn2.ssm_fwd(d["x"], d["dt"], d["B"], d["C"], d["A"], d["D"], d["dt_bias"], d["s0"])
    y = torch.full_like(ref[0], float("nan"))
    state = d["s0"].clone()
    got = gdn2.ssm_fwd(x, dt, b, c, d["A"], d["D"], d["dt_bias"], state, y=y, final_state=state)
    assert got[0] is y and got[1] is state
    assert torch.equal(y, ref[0]) and torch.equal(state, ref[1])


def packed_case(dtype, lengths, H, G, dk, dv, seed, lead=0, behind=0):
    total = lead + sum(lengths) + behind
    k = scan_case(dtype, (total,), H, G, dk, dv, seed, len(lengths))
    cu = [lead]
    for n in lengths:
        cu.append(cu[-1] + n)
    return k, torch.tensor(cu, dtype=torch.int64)


@pytest.mark.parametrize("dtype,dk,dv", [(BF16, 128, 64), (BF16, 64, 128), (F32, 64, 64), (F32, 128, 128)])
def test_packed_scan_matches_oracle(dtype, dk, dv):
    """Lengths of zero, one, and about a chunk; tokens before the first and behind the last
    sequence keep what y held, whatever their inputs are."""
    lengths = [0, 1, 64, 63, 0, 65, 200, 2, 0]
    k, cu = packed_case(dtype, lengths, 4, 2, dk, dv, 7, lead=3, behind=5)
    end = int(cu[-1])
    for n in ("x", "dt", "B", "C"):
        k[n][:3] = float("nan")
        k[n][end:] = float("inf")
    d = dev(k)
    y0 = torch.full((end + 5, 4, dv), 7.0, dtype=dtype, device="cuda")
    y, s = gdn2.ssm_fwd_varlen(d["x"], d["dt"], d["B"], d["C"], d["A"], cu.cuda(), d["D"], d["dt_bias"], d["s0"], y=y0)
    assert y is y0 and (y[:3] == 7).all() and (y[end:] == 7).all()
    for i, n in enumerate(lengths):
        if n == 0:
            assert torch.equal(s[i].cpu(), k["s0"][i])
            continue
        lo = int(cu[i])
        one = {m: (v[None, lo:lo + n] if m in ("x", "dt", "B", "C") else v) for m, v in k.items()}
        one["s0"] = k["s0"][i:i + 1]
        check_scan(one, y[None, lo:lo + n], s[i:i + 1], oracle_scan(one), (n + 63) // 64)


@pytest.mark.parametrize("dtype,H,G,dk,dv,in_place", [(BF16, 2, 1, 128, 128, True), (BF16, 4, 2, 64, 64, False),
                                                      (F32, 1, 1, 64, 64, True)])
def test_packed_scan_cut_into_segments(dtype, H, G, dk, dv, in_place):
    """Sequences around one and several segments, an empty one among them; the same call without a
    workspace walks them whole and agrees within both bars."""
    lengths = [0, 256, 257, 1, 1500, 700, 512, 0, 3]
    k, cu = packed_case(dtype, lengths, H, G, dk, dv, 17, lead=1, behind=2)
    assert gdn2.ssm_fwd_varlen_workspace_bytes(len(lengths), sum(lengths) + 3, H, dk, dv, dtype) > 0
    d = dev(k)
    state = d["s0"].clone()
    y, s = gdn2.ssm_fwd_varlen(d["x"], d["dt"], d["B"], d["C"], d["A"], cu.cuda(), d["D"], d["dt_bias"], state,
                               final_state=state if in_place else None)
    again, s2 = gdn2.ssm_fwd_varlen(d["x"], d["dt"], d["B"], d["C"], d["A"], cu.cuda(), d["D"], d["dt_bias"], d["s0"])
    inside = slice(1, int(cu[-1]))
    assert torch.equal(y[inside], again[inside]) and torch.equal(s, s2)
    for i, n in enumerate(lengths):
        if n == 0:
            assert torch.equal(s[i].cpu(), k["s0"][i])
            continue
        lo = int(cu[i])
        one = {m: (v[None, lo:lo + n] if m in ("x", "dt", "B", "C") else v) for m, v in k.items()}
        one["s0"] = k["s0"][i:i + 1]
        check_scan(one, y[None, lo:lo + n], s[i:i + 1], oracle_scan(one), (n + 63) // 64)


@pytest.mark.parametrize("dtype,T", [(BF16, 1600), (F32, 333), (BF16, 3300)])
def test_scan_forms_the_same_starts_in_place(dtype, T):
    """Few segments form their starts themselves, unless the final state takes the initial one's
    place (then, and for many segments, a pass of its own does)."""
    k = scan_case(dtype, (2, T), 2, 1, 64, 64, 29, 2)
    d = dev(k)
    assert gdn2.ssm_fwd_workspace_bytes(2, T, 2, 64, 64, dtype) > 0
    args = (d["x"], d["dt"], d["B"], d["C"], d["A"], d["D"], d["dt_bias"])
    y, s = gdn2.ssm_fwd(*args, d["s0"])
    check_scan(k, y, s, oracle_scan(k), (T + 63) // 64)
    state = d["s0"].clone()
    y2, s2 = gdn2.ssm_fwd(*args, state, final_state=state)
    assert torch.equal(y, y2) and torch.equal(s, s2)
    zero = torch.zeros_like(state)
    y3, s3 = gdn2.ssm_fwd(*args, None)
    y4, s4 = gdn2.ssm_fwd(*args, zero, final_state=zero)
    assert torch.equal(y3, y4) and torch.equal(s3, s4)


def test_packed_scan_with_few_and_many_segments():
    lengths = [2300, 300, 1700, 0, 900, 5]
    k, cu = packed_case(BF16, lengths, 2, 1, 64, 128, 31)
    d = dev(k)
    args = (d["x"], d["dt"], d["B"], d["C"], d["A"], cu.cuda(), d["D"], d["dt_bias"])
    y, s = gdn2.ssm_fwd_varlen(*args, d["s0"])
    state = d["s0"].clone()
    y2, s2 = gdn2.ssm_fwd_varlen(*args, state, final_state=state)
    assert torch.equal(y, y2) and torch.equal(s, s2)
    for i, n in enumerate(lengths):
        lo = int(cu[i])
        one = {m: (v[None, lo:lo + n] if m in ("x", "dt", "B", "C") else v) for m, v in k.items()}
        one["s0"] = k["s0"][i:i + 1]
        if n:
            check_scan(one, y[None, lo:lo + n], s[i:i + 1], oracle_scan(one), (n + 63) // 64)


@pytest.mark.parametrize("N", [600, 2500])
def test_packed_scan_of_many_sequences(N):
    """More sequences than the order by length is kept for, and more than a workgroup's threads; a few
    long ones are cut."""
    g = torch.Generator("cpu").manual_seed(N)
    lengths = torch.randint(0, 9, (N,), generator=g).tolist()
    lengths[7], lengths[N - 1] = 1100, 400
    k, cu = packed_case(BF16, lengths, 1, 1, 64, 64, 18)
    d = dev(k)
    y, s = gdn2.ssm_fwd_varlen(d["x"], d["dt"], d["B"], d["C"], d["A"], cu.cuda(), d["D"], d["dt_bias"], d["s0"])
    for i in [0, 7, 8, 511, 512, N - 2, N - 1]:
        lo, n = int(cu[i]), lengths[i]
        if n == 0:
            assert torch.equal(s[i].cpu(), k["s0"][i])
            continue
        one = {m: (v[None, lo:lo + n] if m in ("x", "dt", "B", "C") else v) for m, v in k.items()}
        one["s0"] = k["s0"][i:i + 1]
        check_scan(one, y[None, lo:lo + n], s[i:i + 1], oracle_scan(one), (n + 63) // 64)


def test_packed_scan_of_equal_lengths_is_the_scan():
    k = scan_case(BF16, (3, 130), 2, 1, 128, 128, 8, 3)
    d = dev(k)
    y, s = gdn2.ssm_fwd(d["x"], d["dt"], d["B"], d["C"], d["A"], d["D"], d["dt_bias"], d["s0"])
    f = {n: d[n].flatten(0, 1) for n in ("x", "dt", "B", "C")}
    cu = torch.tensor([0, 130, 260, 390], device="cuda")
    yp, sp = gdn2.ssm_fwd_varlen(f["x"], f["dt"], f["B"], f["C"], d["A"], cu, d["D"], d["dt_bias"], d["s0"])
    assert torch.equal(yp.reshape(y.shape), y) and torch.equal(sp, s)


def test_packed_scan_of_no_tokens_and_of_offsets_outside():
    """No tokens at all hands the states on; ranges are clamped into the tensor."""
    k, cu = packed_case(F32, [4, 6], 2, 1, 64, 64, 9)
    d = dev(k)
    none = {n: d[n][:0] for n in ("x", "dt", "B", "C")}
    y, s = gdn2.ssm_fwd_varlen(none["x"], none["dt"], none["B"], none["C"], d["A"],
                               torch.zeros(3, dtype=torch.int64, device="cuda"), d["D"], d["dt_bias"], d["s0"])
    assert y.shape == (0, 2, 64) and torch.equal(s, d["s0"])
    args = (d["x"], d["dt"], d["B"], d["C"], d["A"])
    rest = (d["D"], d["dt_bias"], d["s0"])
    ref = gdn2.ssm_fwd_varlen(*args, torch.tensor([0, 4, 10], device="cuda"), *rest)
    got = gdn2.ssm_fwd_varlen(*args, torch.tensor([-50, 4, 1 << 40], device="cuda"), *rest)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])


@pytest.mark.parametrize("dtype,N,H,G,dk,dv", [(BF16, 5, 4, 2, 128, 128), (BF16, 1, 3, 1, 64, 128),
                                               (F32, 7, 2, 2, 128, 64), (F32, 2, 2, 1, 64, 64)])
def test_step_matches_oracle(dtype, N, H, G, dk, dv):
    """Four steps in a row, each held to the oracle on the state that it began with."""
    say("case: step %s N%d H%d dk%d dv%d" % (dtype, N, H, dk, dv))
    k = scan_case(dtype, (N, 4), H, G, dk, dv, 13 + N, N)
    state = k["s0"].cuda()
    for t in range(4):
        one = {n: (v[:, t:t + 1] if n in ("x", "dt", "B", "C") else v) for n, v in k.items()}
        one["s0"] = state.cpu()
        d = dev(k)
        y = gdn2.ssm_step(*(d[n][:, t] for n in ("x", "dt", "B", "C")), d["A"], state, d["D"], d["dt_bias"])
        yr, sr, ya, sa = oracle_scan(one)
        dx = np.abs(f64(k["D"])[:, None] * f64(one["x"]))
        tol = 320 * U * (ya + dx) + (2.0 ** -8 * np.abs(yr) if dtype == BF16 else 0)
        within("y", y[:, None], yr, tol)
        within("state", state, sr, 320 * U * sa)


# ---- convolution ----------------------------------------------------------------------------

def conv_case(dtype, lead, C, n, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    return dict(x=r(*lead, C).to(dtype), taps=r(C, 4), bias=r(C), s0=r(n, 3, C).to(dtype))


def conv_ref(x, taps, bias, s0):
    """y, the bar of y, and the inputs kept, of [B,T,C]."""
    y, kept = O.short_conv(x, taps, bias, s0)
    ab = lambda t: None if t is None else np.abs(f64(t))
    xa, ta, ba, sa = ab(x), ab(taps), ab(bias), ab(s0)
    B, T, C = xa.shape
    row = np.concatenate([np.zeros((B, 3, C)) if sa is None else sa, xa], 1)
    ua = sum(ta[:, j] * row[:, j:j + T] for j in range(4)) + (0 if ba is None else ba)
    tol = 1.1 * 8 * U * ua + (8 + 4 * ua) * U * np.abs(y)
    if x.dtype == BF16:
        tol = tol + 2.0 ** -8 * np.abs(y)
    return y, tol, kept


@pytest.mark.parametrize("dtype,B,T,C", [(BF16, 2, 1, 8), (BF16, 3, 2, 72), (BF16, 2, 130, 320), (BF16, 1, 37, 2304),
                                         (F32, 2, 3, 8), (F32, 1, 65, 136), (F32, 2, 100, 256)])
def test_conv_matches_oracle(dtype, B, T, C):
    say("case: conv %s B%d T%d C%d" % (dtype, B, T, C))
    k = conv_case(dtype, (B, T), C, B, T + C)
    d = dev(k)
    for bias, s0 in ((None, None), (d["bias"], d["s0"])):
        y, kept = gdn2.short_conv(d["x"], d["taps"], bias, s0)
        ref, tol, kr = conv_ref(k["x"], k["taps"], None if bias is None else k["bias"], None if s0 is None else k["s0"])
        within("y", y, ref, tol)
        assert np.array_equal(f64(kept), kr)
    state = d["s0"].clone()
    y2, same = gdn2.short_conv(d["x"], d["taps"], d["bias"], state, final_state=state)
    assert same is state and torch.equal(y2, y) and torch.equal(state, kept)
    y3, none = gdn2.short_conv(d["x"], d["taps"], d["bias"], d["s0"], output_final_state=False)
    assert none is None and torch.equal(y3, y)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("in_place", [False, True])
def test_packed_conv_matches_oracle(dtype, in_place):
    lengths = [0, 1, 2, 3, 0, 0, 17, 40, 16, 15, 1, 1, 64, 0]
    C, lead, behind = 136, 2, 9
    total = lead + sum(lengths) + behind
    k = conv_case(dtype, (total,), C, len(lengths), 21)
    cu = torch.tensor([lead] + [lead + sum(lengths[:i + 1]) for i in range(len(lengths))])
    end = int(cu[-1])
    k["x"][:lead] = float("nan")
    k["x"][end:] = float("nan")
    wide = torch.cat([k["x"], k["x"]], -1).cuda()  # a token stride of its own
    d = dev(k)
    y0 = torch.full((total, C), 7.0, dtype=dtype, device="cuda")
    out = d["s0"] if in_place else torch.full_like(d["s0"], float("nan"))
    y, kept = gdn2.short_conv_varlen(wide[:, C:], d["taps"], cu.cuda(), d["bias"], d["s0"], y=y0, final_state=out)
    assert y is y0 and kept is out and (y[:lead] == 7).all() and (y[end:] == 7).all()
    for i, n in enumerate(lengths):
        lo = int(cu[i])
        ref, tol, kr = conv_ref(k["x"][None, lo:lo + n], k["taps"], k["bias"], k["s0"][i:i + 1])
        assert np.array_equal(f64(kept[i:i + 1]), kr), i
        if n:
            within("seq %d" % i, y[None, lo:lo + n], ref, tol)


@pytest.mark.parametrize("dtype,N,C", [(BF16, 5, 72), (F32, 3, 264), (BF16, 1, 2304)])
def test_conv_step_matches_prompt(dtype, N, C):
    k = conv_case(dtype, (N, 6), C, N, 31)
    d = dev(k)
    y, kept = gdn2.short_conv(d["x"], d["taps"], d["bias"], d["s0"])
    state = d["s0"].clone()
    for t in range(6):
        yt = gdn2.short_conv_step(d["x"][:, t], d["taps"], state, d["bias"])
        ref, tol, _ = conv_ref(k["x"][:, :t + 1], k["taps"], k["bias"], k["s0"])
        within("token %d" % t, yt, ref[:, t], tol[:, t])
    assert torch.equal(state, kept)


# ---- norm -----------------------------------------------------------------------------------

def norm_bars(x, g, b, y, mean, rstd, dtype):
    m = np.abs(x).mean(-1)
    xh = (x - mean[:, None]) * rstd[:, None]
    tol = np.abs(g) * (rstd * 100 * U * m)[:, None] + 125 * U * np.abs(g * xh) + 4 * U * (np.abs(y) + np.abs(b))
    return tol + (2.0 ** -8 * np.abs(y) if dtype == BF16 else 0), 100 * U * m, 125 * U * rstd


NORMS = [(1, 1), (3, 2), (5, 7), (2, 8), (130, 64), (33, 100), (1, 2048), (70, 1000), (9, 1537), (4, 2056), (3, 4099),
         (2, 8192), (2, 16384), (3, 16383), (1001, 257)]


def norm_case(dtype, rows, width, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    x = torch.randn(rows, width, generator=g) * 2 + torch.randn(rows, 1, generator=g) * 3
    if rows > 2:
        x[1] = 3.3  # a row without variance
    return dict(x=x.to(dtype), gamma=torch.randn(width, generator=g), beta=torch.randn(width, generator=g),
                dy=torch.randn(rows, width, generator=g).to(dtype))


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,width", NORMS)
def test_norm_and_its_gradients_match_oracle(dtype, rows, width):
    say("case: norm %s %d x %d" % (dtype, rows, width))
    k = norm_case(dtype, rows, width, rows + width)
    d = dev(k)
    x, g, b, dy = (f64(k[n]) for n in ("x", "gamma", "beta", "dy"))
    for beta in (d["beta"], None):
        y, mean, rstd = gdn2.layer_norm(d["x"], d["gamma"], beta, 1e-5)
        bb = b if beta is not None else 0 * b
        ref, mr, rr = O.layer_norm(x, g, bb, 1e-5)
        ty, tm, tr = norm_bars(x, g, bb, ref, mr, rr, dtype)
        within("y", y, ref, ty)
        within("mean", mean, mr, tm)
        within("rstd", rstd, rr, tr)
    y2, none, _ = gdn2.layer_norm(d["x"], d["gamma"], None, 1e-5, stats=False)
    assert none is None and torch.equal(y2, y)

    bufs = {"dx": torch.full_like(d["x"], float("nan")), "dgamma": torch.full_like(d["gamma"], float("nan"))}
    out = gdn2.layer_norm_bwd(d["dy"], d["x"], d["gamma"], mean, rstd, grads=bufs)
    assert out["dx"] is bufs["dx"] and out["dgamma"] is bufs["dgamma"]
    m, r = f64(mean), f64(rstd)
    dx, dg, db = O.layer_norm_bwd(dy, x, g, m, r)
    u = np.abs((x - m[:, None]) * r[:, None])
    v = np.abs(dy * g)
    tol = r[:, None] * U * (100 * v.mean(-1)[:, None] + 130 * u * (u * v).mean(-1)[:, None] + 8 * v)
    within("dx", out["dx"], dx, tol + (2.0 ** -8 * np.abs(dx) if dtype == BF16 else 0))
    within("dgamma", out["dgamma"], dg, 600 * U * (np.abs(dy) * u).sum(0))
    within("dbeta", out["dbeta"], db, 600 * U * np.abs(dy).sum(0))
    again = gdn2.layer_norm_bwd(d["dy"], d["x"], d["gamma"], mean, rstd, want_beta_grad=False)
    assert again["dbeta"] is None and torch.equal(again["dgamma"], out["dgamma"]) and torch.equal(again["dx"], out["dx"])


def test_norm_gradients_against_differences():
    """The kernels' own outputs, fp32: dgamma, dbeta and dx times a direction against the change
    of sum(dy y) along it.  The differences' error: y's bar summed over the step's two ends, and
    the cubic term, which a step of 1e-2 keeps at 1e-4 of the sum of sizes."""
    k = norm_case(F32, 6, 200, 77)
    k["x"][1] = k["x"][0] * 0.5 - 1
    d = dev(k)
    y, mean, rstd = gdn2.layer_norm(d["x"], d["gamma"], d["beta"])
    out = gdn2.layer_norm_bwd(d["dy"], d["x"], d["gamma"], mean, rstd)
    h = 1e-2
    for name, grad in (("x", "dx"), ("gamma", "dgamma"), ("beta", "dbeta")):
        way = torch.randn(d[name].shape, generator=torch.Generator("cpu").manual_seed(5)).cuda()
        ends = [{**d, name: d[name] + s * h * way} for s in (1, -1)]
        f = [(d["dy"].double() * gdn2.layer_norm(e["x"], e["gamma"], e["beta"])[0].double()).sum() for e in ends]
        size = float((out[grad].double() * way.double()).abs().sum())
        slope = float((f[0] - f[1]) / (2 * h))
        noise = float(d["dy"].abs().sum()) * 8 * 200 * U / h
        assert abs(slope - float((out[grad].double() * way.double()).sum())) <= 1e-4 * size + noise, name


def test_norm_of_no_rows():
    g = torch.ones(40, device="cuda")
    x = torch.empty(0, 40, device="cuda")
    y, mean, rstd = gdn2.layer_norm(x, g)
    assert y.shape == (0, 40) and mean.shape == (0,)
    out = gdn2.layer_norm_bwd(x, x, g, mean, rstd, grads={"dgamma": torch.full_like(g, 3.0)})
    assert (out["dgamma"] == 0).all() and (out["dbeta"] == 0).all()


# ---- together -------------------------------------------------------------------------------

def block_weights(width, H, G, dk, dv, seed):
    g = torch.Generator("cpu").manual_seed(seed)
    r = lambda *s: torch.randn(s, generator=g)
    ch = H * dv + 2 * G * dk
    return dev(dict(gamma=1 + 0.1 * r(width), beta=0.1 * r(width), win=r(width, ch + H + H * dv) / width ** 0.5,
                    taps=0.5 * r(ch, 4), bias=0.1 * r(ch), A=-torch.rand(H, generator=g) * 8 - 1, D=r(H),
                    dt_bias=r(H) - 4, out_gamma=1 + 0.1 * r(dv)))


def split_projection(p, H, G, dk, dv):
    xbc, dt, z = p.split([H * dv + 2 * G * dk, H, H * dv], -1)
    return xbc, dt, z


def test_block_prompts_then_tokens():
    """Packed prompts through norm, projection, convolution, scan and the gated output norm, then
    two tokens of each sequence from the states kept: the tokens' outputs are those of the longer
    prompts.  The two roads differ in where bf16 rounds: y is off by 2^-8 of its terms on each, so
    4 parts of 2^-8 of their sum of sizes bound the difference of the scans' outputs, with the
    same inputs (the projection is computed once, in fp32, and rounded)."""
    H, G, dk, dv, width = 4, 2, 64, 64, 96
    w = block_weights(width, H, G, dk, dv, 3)
    lengths = [5, 70, 1, 130]
    full = [n + 2 for n in lengths]
    g = torch.Generator("cpu").manual_seed(4)
    h = torch.randn(sum(full), width, generator=g).to(BF16).cuda()
    hn, _, _ = gdn2.layer_norm(h, w["gamma"], w["beta"], stats=False)
    p = (hn.float() @ w["win"]).to(BF16)
    starts = np.cumsum([0] + full)

    def prompts(rows, lens):
        cu = torch.tensor(np.cumsum([0] + lens), device="cuda")
        xbc, dt, z = split_projection(p[rows], H, G, dk, dv)
        u, kept = gdn2.short_conv_varlen(xbc, w["taps"], cu, w["bias"])
        x, b, c = u.split([H * dv, G * dk, G * dk], -1)
        x, b, c = x.unflatten(-1, (H, dv)), b.unflatten(-1, (G, dk)), c.unflatten(-1, (G, dk))
        y, s = gdn2.ssm_fwd_varlen(x, dt, b, c, w["A"], cu, w["D"], w["dt_bias"])
        o = gdn2.mixer_out(y[None], z.contiguous().unflatten(-1, (H, dv))[None], w["out_gamma"])
        return y, o[0], kept, s, (x, dt, b, c)

    every = torch.arange(sum(full))
    y_all, o_all, kept_all, s_all, ins = prompts(every, full)
    rows = torch.cat([every[starts[i]:starts[i] + n] for i, n in enumerate(lengths)])
    _, _, kept, s, _ = prompts(rows, lengths)
    for t in range(2):
        at = torch.tensor([starts[i] + n + t for i, n in enumerate(lengths)])
        xbc, dt, z = split_projection(p[at], H, G, dk, dv)
        u = gdn2.short_conv_step(xbc, w["taps"], kept, w["bias"])
        x, b, c = u.split([H * dv, G * dk, G * dk], -1)
        y = gdn2.ssm_step(x.unflatten(-1, (H, dv)), dt, b.unflatten(-1, (G, dk)), c.unflatten(-1, (G, dk)), w["A"], s,
                          w["D"], w["dt_bias"])
        o = gdn2.mixer_out(y[:, None], z.contiguous().unflatten(-1, (H, dv))[:, None], w["out_gamma"])
        assert torch.isfinite(o).all()
        for i in range(len(lengths)):
            lo, hi = starts[i], starts[i] + lengths[i] + t + 1
            k = dict(zip(("x", "dt", "B", "C"), (v[None, lo:hi] for v in ins)), A=w["A"], D=w["D"], dt_bias=w["dt_bias"], s0=None)
            yr, _, ya, _ = oracle_scan(k)
            tol = 2.0 ** -8 * (1 + 2.0 ** -7) * ya[:, -1] + 2.0 ** -8 * np.abs(yr[:, -1]) + 400 * U * ya[:, -1]
            tol = tol + 400 * U * np.abs(f64(w["D"])[:, None] * f64(k["x"])[:, -1])
            within("token", y[i][None], yr[:, -1], tol)
            within("prompt", y_all[at[i]][None], yr[:, -1], tol)
    assert torch.equal(kept, kept_all)


def test_norm_layer_training_step_uses_the_gradients():
    """One descent step through norm and a projection lowers nothing by itself here: the gradient
    of the projection's input, carried through layer_norm_bwd, is the fp64 chain's."""
    rows, width, out = 37, 120, 24
    k = norm_case(F32, rows, width, 9)
    g = torch.Generator("cpu").manual_seed(10)
    wp, dz = torch.randn(width, out, generator=g), torch.randn(rows, out, generator=g)
    d = dev(k)
    y, mean, rstd = gdn2.layer_norm(d["x"], d["gamma"], d["beta"])
    dy = (dz.double() @ wp.double().T).float()
    grads = gdn2.layer_norm_bwd(dy.cuda(), d["x"], d["gamma"], mean, rstd)
    x, gm, bt = (k[n].double().requires_grad_() for n in ("x", "gamma", "beta"))
    m = x.mean(-1, keepdim=True)
    ref = ((x - m) / ((x - m).square().mean(-1, keepdim=True) + 1e-5).sqrt() * gm + bt) @ wp.double()
    (ref * dz.double()).sum().backward()
    r = f64(rstd)[:, None]
    u = np.abs((f64(k["x"]) - f64(mean)[:, None]) * r)
    v = np.abs(f64(dy) * f64(k["gamma"]))
    tol = r * U * (200 * v.mean(-1)[:, None] + 400 * u * (u * v).mean(-1)[:, None] + 200 * v)
    keep = np.arange(rows) != 1  # the row without variance: rstd's own error is the whole of it
    within("dx", grads["dx"][torch.from_numpy(keep)], x.grad.numpy()[keep], tol[keep])
    within("dgamma", grads["dgamma"], gm.grad.numpy(), 900 * U * (np.abs(f64(dy)) * (u + 1)).sum(0))
    within("dbeta", grads["dbeta"], bt.grad.numpy(), 900 * U * np.abs(f64(dy)).sum(0))


# ---- streams and graphs ---------------------------------------------------------------------

def test_calls_on_another_stream():
    k = scan_case(BF16, (1, 2500), 2, 1, 128, 64, 40, 1)
    d = dev(k)
    ref = gdn2.ssm_fwd(d["x"], d["dt"], d["B"], d["C"], d["A"], d["D"], d["dt_bias"], d["s0"])
    nk = dev(norm_case(BF16, 300, 500, 41))
    nref = gdn2.layer_norm(nk["x"], nk["gamma"], nk["beta"])
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = gdn2.ssm_fwd(d["x"], d["dt"], d["B"], d["C"], d["A"], d["D"], d["dt_bias"], d["s0"])
        ngot = gdn2.layer_norm(nk["x"], nk["gamma"], nk["beta"])
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref + nref, got + ngot))


def test_two_graphs_replayed_in_turn():
    """Each graph holds a scan in segments, a packed convolution in place, a step and norm
    gradients, on its own inputs; replays of the two alternate, with eager work between."""
    def make(seed):
        k = dev(scan_case(BF16, (1, 2300), 2, 1, 64, 64, seed, 1))
        c = dev(conv_case(BF16, (50,), 64, 3, seed))
        n = dev(norm_case(BF16, 400, 300, seed))
        st = dev(scan_case(F32, (4,), 2, 1, 64, 128, seed, 4))
        cu = torch.tensor([0, 20, 21, 50], device="cuda")

        def go():
            y, s = gdn2.ssm_fwd(k["x"], k["dt"], k["B"], k["C"], k["A"], k["D"], k["dt_bias"], k["s0"])
            kept = c["s0"].clone()
            u, _ = gdn2.short_conv_varlen(c["x"], c["taps"], cu, c["bias"], kept, final_state=kept)
            state = st["s0"].clone()
            t = gdn2.ssm_step(st["x"], st["dt"], st["B"], st["C"], st["A"], state, st["D"], st["dt_bias"])
            v, mean, rstd = gdn2.layer_norm(n["x"], n["gamma"], n["beta"])
            gr = gdn2.layer_norm_bwd(n["dy"], n["x"], n["gamma"], mean, rstd)
            return [y, s, u, kept, t, state, v, mean, rstd, gr["dx"], gr["dgamma"], gr["dbeta"]]
        return go

    makers = [make(50), make(51)]
    refs = [[t.clone() for t in go()] for go in makers]
    torch.cuda.synchronize()
    graphs = []
    for go in makers:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs = go()
        graphs.append((g, outs))
    for _ in range(3):
        for i in (0, 1):
            for t in graphs[i][1]:
                t.fill_(-9.0)
            graphs[i][0].replay()
            makers[1 - i]()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(graphs[i][1], refs[i]))


# ---- sizes past 32 bits ---------------------------------------------------------------------

def test_scan_past_32_bit_offsets():
    """2.3e9 elements (4.6 GB) of x: the last sequences give what they give alone."""
    N, T, H, G, dk, dv = 17600, 64, 32, 1, 64, 64
    k = dev(scan_case(BF16, (16, T), H, G, dk, dv, 60))
    x = torch.zeros(N, T, H, dv, dtype=BF16, device="cuda")
    dt = torch.zeros(N, T, H, dtype=BF16, device="cuda")
    B = torch.zeros(N, T, G, dk, dtype=BF16, device="cuda")
    C = torch.zeros_like(B)
    assert x.numel() > 2 ** 31
    for big, name in ((x, "x"), (dt, "dt"), (B, "B"), (C, "C")):
        big[-16:] = k[name]
    rest = (k["A"], k["D"], k["dt_bias"])
    ref, sref = gdn2.ssm_fwd(k["x"], k["dt"], k["B"], k["C"], *rest)
    y, s = gdn2.ssm_fwd(x, dt, B, C, *rest)
    assert torch.equal(y[-16:], ref) and torch.equal(s[-16:], sref)
    assert not y[:16].any() and not s[:16].any()
    y.fill_(7)
    cu = (torch.arange(N + 1) * T).cuda()
    gdn2.ssm_fwd_varlen(x.flatten(0, 1), dt.flatten(0, 1), B.flatten(0, 1), C.flatten(0, 1), k["A"], cu, k["D"],
                        k["dt_bias"], y=y.flatten(0, 1), final_state=s)
    assert torch.equal(y[-16:], ref) and torch.equal(s[-16:], sref)


def test_conv_and_norm_past_32_bit_offsets():
    rows, width = 281000, 8192
    g = torch.Generator("cpu").manual_seed(61)
    tail = torch.randn(400, width, generator=g).to(BF16).cuda()
    taps, bias, gamma = (torch.randn(s, generator=g).cuda() for s in ((width, 4), (width,), (width,)))
    x = torch.zeros(rows, width, dtype=BF16, device="cuda")
    assert x.numel() > 2 ** 31
    x[-400:] = tail
    y, kept = gdn2.short_conv(x[None], taps, bias)
    ref, rkept = gdn2.short_conv(tail[None], taps, bias)
    assert torch.equal(y[0, -400:], ref[0]) and torch.equal(kept, rkept)
    cu = torch.tensor([0, 5, rows - 400, rows], device="cuda")
    _, kept = gdn2.short_conv_varlen(x, taps, cu, bias, y=y[0].fill_(7))
    assert torch.equal(y[0, -400:], ref[0]) and torch.equal(kept[2:], rkept)
    y, mean, rstd = gdn2.layer_norm(x, gamma, y=y[0])
    ref, rmean, rrstd = gdn2.layer_norm(tail, gamma)
    assert torch.equal(y[-400:], ref) and torch.equal(mean[-400:], rmean) and torch.equal(rstd[-400:], rrstd)
    # rows of zeros have dy = x = 0 here: only the last ones add to the sums
    got = gdn2.layer_norm_bwd(x, x, gamma, mean, rstd, grads={"dx": y})
    want = gdn2.layer_norm_bwd(tail, tail, gamma, rmean, rrstd)
    assert torch.equal(got["dx"][-400:], want["dx"])
    ab = (tail.double() * (tail.double() - rmean.double()[:, None]) * rrstd.double()[:, None]).abs().sum(0)
    within("dgamma", got["dgamma"], f64(want["dgamma"]), 600 * U * f64(ab))
    within("dbeta", got["dbeta"], f64(want["dbeta"]), 600 * U * f64(tail.double().abs().sum(0)))
