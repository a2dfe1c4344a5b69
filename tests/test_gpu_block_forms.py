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
from oracle import block as O
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


def whole(name, d, sizes, strides, y, s, code, *cu):
    """The library's call without a workspace."""
    ptrs = [t.data_ptr() for t in args_of(d)] + [d["D"].data_ptr(), d["dt_bias"].data_ptr(), d["s0"].data_ptr()]
    block._launch(name, y.device, *ptrs, y.data_ptr(), s.data_ptr(), *cu, *sizes, *strides, code, 1, None, 0)


@pytest.mark.parametrize("dtype,H,G,dk,dv", [(BF16, 2, 1, 128, 128), (F32, 4, 2, 64, 64), (BF16, 32, 2, 64, 64)])
def test_scan_without_a_workspace(dtype, H, G, dk, dv):
    """Sequences that would be cut, walked whole."""
    B, T = 2, 900
    k = scan_case(dtype, (B, T), H, G, dk, dv, 400 + H, B)
    assert gdn2.ssm_fwd_workspace_bytes(B, T, H, dk, dv, dtype) > 0
    d = dev(k)
    y, s = torch.empty_like(d["x"]), torch.empty_like(d["s0"])
    sizes, strides = (B, T, H, G, dk, dv), (H * dv, H, G * dk, G * dk)
    whole("gdn2_ssm_fwd", d, sizes, strides, y, s, 1 if dtype == BF16 else 0)
    for n in range(B):
        one = sequence(k, n)
        check_scan(one, y[n:n + 1], s[n:n + 1], oracle_scan(one), (T + 63) // 64)


@pytest.mark.parametrize("dtype,H,G,dk,dv", [(BF16, 2, 1, 128, 128), (F32, 4, 2, 64, 64), (BF16, 128, 2, 64, 64)])
def test_packed_scan_without_a_workspace(dtype, H, G, dk, dv):
    lengths = [0, 256, 257, 1, 900, 700, 512, 0, 3]
    k, cu = packed_case(dtype, lengths, H, G, dk, dv, 410 + H)
    assert gdn2.ssm_fwd_varlen_workspace_bytes(len(lengths), sum(lengths), H, dk, dv, dtype) > 0
    d = dev(k)
    y, s = torch.empty_like(d["x"]), torch.empty_like(d["s0"])
    at = cu.cuda()
    sizes, strides = (len(lengths), sum(lengths), H, G, dk, dv), (H * dv, H, G * dk, G * dk)
    whole("gdn2_ssm_fwd_varlen", d, sizes, strides, y, s, 1 if dtype == BF16 else 0, at.data_ptr())
    for n, length in enumerate(lengths):
        if length == 0:
            assert torch.equal(s[n].cpu(), k["s0"][n])
        elif H < 64 or n < 4:
            one = part(k, cu, n)
            check_scan(one, y[None, int(cu[n]):int(cu[n + 1])], s[n:n + 1], oracle_scan(one), (length + 63) // 64)


def guarded(need, align):
    """A caller's workspace at an odd address, and the check that the bytes around it stay."""
    buf = torch.full((need + align + 1024,), 0xAB, dtype=torch.uint8, device="cuda")
    ws = buf[513:513 + need + align]
    lo = 513 + -ws.data_ptr() % align

    def untouched():
        assert (buf[:lo] == 0xAB).all() and (buf[lo + need:] == 0xAB).all()
    return ws, untouched


@pytest.mark.parametrize("dtype,T", [(BF16, 1600), (BF16, 3300), (F32, 333)])
def test_scan_stays_in_the_callers_workspace(dtype, T):
    k = scan_case(dtype, (2, T), 2, 1, 64, 128, 420 + T, 2)
    d = dev(k)
    need = gdn2.ssm_fwd_workspace_bytes(2, T, 2, 64, 128, dtype)
    assert need > 0
    ws, untouched = guarded(need, 256)
    ref = gdn2.ssm_fwd(*args_of(d), d["D"], d["dt_bias"], d["s0"])
    got = gdn2.ssm_fwd(*args_of(d), d["D"], d["dt_bias"], d["s0"], workspace=ws)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    untouched()


@pytest.mark.parametrize("lengths", [[700, 0, 300, 2300, 1, 64], [4] * 700 + [600], [260] * 5])
def test_packed_scan_stays_in_the_callers_workspace(lengths):
    k, cu = packed_case(BF16, lengths, 2, 1, 64, 64, 430 + len(lengths))
    d = dev(k)
    need = gdn2.ssm_fwd_varlen_workspace_bytes(len(lengths), sum(lengths), 2, 64, 64, BF16)
    assert need > 0
    ws, untouched = guarded(need, 256)
    ref = gdn2.ssm_fwd_varlen(*args_of(d), cu.cuda(), d["D"], d["dt_bias"], d["s0"])
    got = gdn2.ssm_fwd_varlen(*args_of(d), cu.cuda(), d["D"], d["dt_bias"], d["s0"], workspace=ws)
    assert torch.equal(ref[0], got[0]) and torch.equal(ref[1], got[1])
    untouched()


@pytest.mark.parametrize("N", [8, 1500])
def test_packed_scan_of_offsets_that_overlap(N):
    """Every second sequence is all of the tokens: more pieces than sequences side by side have.  All
    of them agree with the oracle, those that are cut and those for which the lists have no place."""
    T = 1500 if N == 8 else 300
    k = scan_case(BF16, (T,), 2, 1, 64, 64, 440, None)
    d = dev(k)
    cu = torch.tensor([0, T] * (N // 2) + [0], device="cuda")
    need = gdn2.ssm_fwd_varlen_workspace_bytes(N, T, 2, 64, 64, BF16)
    assert need > 0
    ws, untouched = guarded(need, 256)
    y, s = gdn2.ssm_fwd_varlen(*args_of(d), cu, d["D"], d["dt_bias"], workspace=ws)
    untouched()
    one = {m: (v[None] if m in TOKENS else v) for m, v in k.items()}
    ref = oracle_scan(one)
    for n in (0, 2, N - 2):
        check_scan(one, y[None], s[n:n + 1], ref, (T + 63) // 64)
    assert not s[1::2].any()


def test_packed_scan_writes_states_past_32_bit_offsets():
    """2.3e9 elements of states, of no defined value before the call."""
    N, T, H, G, dk, dv = 17600, 2, 32, 1, 64, 64
    k = scan_case(BF16, (16 * T,), H, G, dk, dv, 450)
    d = dev(k)
    big = {n: torch.zeros(N * T, *d[n].shape[1:], dtype=BF16, device="cuda") for n in TOKENS}
    for n in TOKENS:
        big[n][-16 * T:] = d[n]
    s = torch.full((N, H, dk, dv), float("nan"), device="cuda")
    assert s.numel() > 2 ** 31
    cu = (torch.arange(N + 1) * T).cuda()
    y, _ = gdn2.ssm_fwd_varlen(big["x"], big["dt"], big["B"], big["C"], d["A"], cu, d["D"], d["dt_bias"], final_state=s)
    assert all(not s[lo:lo + 1100].any() for lo in range(0, N - 1100, 1100)) and not s[N - 1100:N - 16].any()
    at = torch.arange(17) * T
    for n in (0, 15):
        one = part(k, at, n)
        lo = (N - 16 + n) * T
        check_scan(one, y[None, lo:lo + T], s[N - 16 + n:N - 15 + n], oracle_scan(one), 1)


# ---- step past the caches -------------------------------------------------------------------

@pytest.mark.parametrize("dtype,N,H,G,dk,dv", [(BF16, 140, 16, 1, 128, 128), (F32, 130, 17, 1, 128, 128),
                                               (BF16, 263, 16, 4, 64, 128), (F32, 270, 16, 2, 128, 64),
                                               (BF16, 530, 16, 8, 64, 64)])
def test_step_past_the_caches_matches_oracle(dtype, N, H, G, dk, dv):
    """More than 128 MB of states: every state and output, against the step's formula in 64 bits."""
    assert N * H * dk * dv * 4 > 128 << 20
    k = scan_case(dtype, (N,), H, G, dk, dv, 500 + N, N)
    d = dev(k)
    state = d["s0"].clone()
    y = gdn2.ssm_step(*args_of(d), state, d["D"], d["dt_bias"])
    x, raw, b, c, a, bias, s0 = (d[n].double() for n in ("x", "dt", "B", "C", "A", "dt_bias", "s0"))
    dt = torch.nn.functional.softplus(raw + bias, threshold=40)
    b, c = b.repeat_interleave(H // G, 1), c.repeat_interleave(H // G, 1)
    keep, put = s0 * torch.exp(dt * a)[..., None, None], (dt[..., None] * b)[..., None] * x[:, :, None]
    s, size = keep + put, keep.abs() + put.abs()
    assert bool(((state.double() - s).abs() <= 320 * U * size + 1e-30).all())
    dx = d["D"].double()[:, None] * x
    want = (s * c[..., None]).sum(-2) + dx
    tol = 320 * U * ((size * c.abs()[..., None]).sum(-2) + dx.abs()) + (2.0 ** -8 * want.abs() if dtype == BF16 else 0)
    assert bool(((y.double() - want).abs() <= tol + 1e-30).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_steps_on_the_last_tokens_of_long_prompts(dtype):
    """[:, -1] of [N, T, C] with T C past 2^22 gives the bits of its copy."""
    N, T, H, G, dk, dv = 3, 2050, 16, 1, 128, 128
    C = H * dv + 2 * G * dk
    assert T * C > 1 << 22
    k = scan_case(dtype, (N,), H, G, dk, dv, 560, N)
    d = dev(k)
    c = dev(conv_case(dtype, (N,), C, N, 561))
    flat = torch.cat([d["x"].flatten(1), d["B"].flatten(1), d["C"].flatten(1)], -1)
    prompts = torch.zeros(N, T, C, dtype=dtype, device="cuda")
    prompts[:, -1] = flat
    steps = torch.zeros(N, T * C, H, dtype=dtype, device="cuda")[:, :1].squeeze(1)
    steps.copy_(d["dt"])
    parts = prompts[:, -1].split([H * dv, G * dk, G * dk], -1)
    far = [v.unflatten(-1, (n, -1)) for v, n in zip(parts, (H, G, G))]
    state, want = d["s0"].clone(), d["s0"].clone()
    ref = gdn2.ssm_step(*args_of(d), want, d["D"], d["dt_bias"])
    got = gdn2.ssm_step(far[0], steps, far[1], far[2], d["A"], state, d["D"], d["dt_bias"])
    assert torch.equal(ref, got) and torch.equal(want, state)
    c["x"] = flat
    kept, want = c["s0"].clone(), c["s0"].clone()
    ref = gdn2.short_conv_step(c["x"], c["taps"], want, c["bias"])
    got = gdn2.short_conv_step(prompts[:, -1], c["taps"], kept, c["bias"])
    assert torch.equal(ref, got) and torch.equal(want, kept)


# ---- convolution in runs of 16 tokens -------------------------------------------------------

@pytest.mark.parametrize("dtype", [BF16, F32])
def test_conv_in_long_runs_matches_oracle(dtype):
    B, T, C = 3, 1201, 2560
    assert B * T // 16 * (C // 4) >= 1 << 17
    k = conv_case(dtype, (B, T), C, B, 600)
    d = dev(k)
    ref, tol, kr = conv_ref(k["x"], k["taps"], k["bias"], k["s0"])
    y, kept = gdn2.short_conv(d["x"], d["taps"], d["bias"], d["s0"])
    within("y", y, ref, tol)
    assert np.array_equal(f64(kept), kr)
    state = d["s0"].clone()
    y2, _ = gdn2.short_conv(d["x"], d["taps"], d["bias"], state, final_state=state)
    assert torch.equal(y, y2) and torch.equal(state, kept)
    ref, tol, _ = conv_ref(k["x"][:1], k["taps"], None, None)
    within("y", gdn2.short_conv(d["x"], d["taps"])[0][:1], ref, tol)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("in_place", [False, True])
def test_packed_conv_in_long_runs_matches_oracle(dtype, in_place):
    """Several short sequences in a run, empty ones, and long ones that begin and end on and beside a run's edges."""
    g = torch.Generator("cpu").manual_seed(610)
    lengths = [16, 16, 15, 17, 1, 0, 0, 2, 3, 10, 0, 333, 1, 400, 31, 33] + torch.randint(0, 30, (120,), generator=g).tolist() + [1000, 16, 0]
    C, lead, behind = 2560, 3, 21
    total = lead + sum(lengths) + behind
    assert total // 16 * (C // 4) >= 1 << 17
    k = conv_case(dtype, (total,), C, len(lengths), 611)
    cu = torch.tensor([lead] + lengths).cumsum(0)
    end = int(cu[-1])
    k["x"][:lead] = float("nan")
    k["x"][end:] = float("nan")
    d = dev(k)
    y0 = torch.full((total, C), 7.0, dtype=dtype, device="cuda")
    out = d["s0"] if in_place else torch.full_like(d["s0"], float("nan"))
    y, kept = gdn2.short_conv_varlen(d["x"], d["taps"], cu.cuda(), d["bias"], d["s0"], y=y0, final_state=out)
    assert (y[:lead] == 7).all() and (y[end:] == 7).all()
    worst = 0.0
    for i, n in enumerate(lengths):
        lo = int(cu[i])
        ref, tol, kr = conv_ref(k["x"][None, lo:lo + n], k["taps"], k["bias"], k["s0"][i:i + 1])
        assert np.array_equal(f64(kept[i:i + 1]), kr), i
        if n:
            worst = max(worst, float((np.abs(f64(y[None, lo:lo + n]) - ref) / (tol + 1e-30)).max()))
    assert worst <= 1.0, worst


# ---- norm -----------------------------------------------------------------------------------

@pytest.mark.parametrize("dtype,rows,width", [(BF16, 300, 1000), (F32, 1001, 1540), (F32, 9, 16384)])
def test_norm_gradients_stay_in_the_callers_workspace(dtype, rows, width):
    g = torch.Generator("cpu").manual_seed(rows)
    x, dy = (torch.randn(rows, width, generator=g).to(dtype).cuda() for _ in range(2))
    gamma = torch.randn(width, generator=g).cuda()
    _, mean, rstd = gdn2.layer_norm(x, gamma)
    need = gdn2.layer_norm_bwd_workspace_bytes(rows, width)
    assert need > 0
    ws, untouched = guarded(need, 16)
    ref = gdn2.layer_norm_bwd(dy, x, gamma, mean, rstd)
    got = gdn2.layer_norm_bwd(dy, x, gamma, mean, rstd, workspace=ws)
    assert all(torch.equal(ref[n], got[n]) for n in ref)
    untouched()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("rows,width", [(1, 1), (4000, 130), (70, 1000), (1001, 1540), (1536, 2048), (300, 4096), (100, 8192),
                                        (3, 16383)])
def test_norm_within_the_roundings_of_its_sums(dtype, rows, width):
    """Bars that count the roundings on the way of a row's sums: 8 elements of a lane (16 above 8192
    columns), six steps over a wave, one a wave of the row, and two of the factor 1 / width; of the
    sums over rows: the rows of a thread, those side by side in a workgroup, and the parts."""
    say("case: norm roundings %s %d x %d" % (dtype, rows, width))
    lanes = 16
    while lanes < 1024 and width > lanes * 8:
        lanes *= 2
    a = (7 if width <= 8192 else 15) + 6 + lanes // 64 + 2
    g = torch.Generator("cpu").manual_seed(rows + width)
    x = (torch.randn(rows, width, generator=g) + torch.randn(rows, 1, generator=g)).to(dtype)
    dy = torch.randn(rows, width, generator=g).to(dtype)
    gamma, beta = torch.randn(width, generator=g), torch.randn(width, generator=g)
    y, mean, rstd = gdn2.layer_norm(x.cuda(), gamma.cuda(), beta.cuda(), 1e-5)
    xd, dyd, gd, bd = (f64(t) for t in (x, dy, gamma, beta))
    yr, mr, rr = O.layer_norm(xd, gd, bd, 1e-5)
    one = 1 + 2.0 ** -15  # the products of roundings
    off = one * a * U * np.abs(xd).mean(-1)
    var = 1 / rr ** 2 - 1e-5
    rel = one * (0.5 * ((a + 4) * U * var + off ** 2 + U / rr ** 2) * rr ** 2 + 3 * U)
    xh = (xd - mr[:, None]) * rr[:, None]
    out = lambda v: 2.0 ** -8 * np.abs(v) if dtype == BF16 else 0
    within("mean", mean, mr, off)
    within("rstd", rstd, rr, rel * rr)
    tol = np.abs(gd) * (rr * off * (1 + rel))[:, None] + np.abs(gd * xh) * (rel[:, None] + 3 * U) + U * (np.abs(yr) + np.abs(bd))
    within("y", y, yr, one * tol + out(yr))

    got = gdn2.layer_norm_bwd(dy.cuda(), x.cuda(), gamma.cuda(), mean, rstd)
    m, r = f64(mean)[:, None], f64(rstd)[:, None]
    dx, dg, db = O.layer_norm_bwd(dyd, xd, gd, m[:, 0], r[:, 0])
    u, v = np.abs((xd - m) * r), np.abs(dyd * gd)
    mv, muv = v.mean(-1, keepdims=True), (u * v).mean(-1, keepdims=True)
    tol = r * U * ((a + 1) * mv + (a + 4) * u * muv + 5 * (v + mv + u * muv))
    within("dx", got["dx"], dx, one * tol + out(dx))
    side = max(1, 256 // lanes)  # rows of a workgroup at once
    groups = -(-rows // side)
    groups = 1 if groups <= 8 else min(groups, 512 if lanes == 1024 else 393216 // max(256, lanes))
    n = -(-rows // (groups * side)) + side + -(-groups // 32) + 5
    within("dgamma", got["dgamma"], dg, one * (n + 4) * U * (np.abs(dyd) * u).sum(0))
    within("dbeta", got["dbeta"], db, one * n * U * np.abs(dyd).sum(0))


# ---- values that are not finite -------------------------------------------------------------

@pytest.mark.parametrize("dtype,B,T,H,G,dk,dv", [
    (BF16, 1, 150, 2, 1, 64, 64), (BF16, 1, 150, 2, 1, 128, 128), (BF16, 9, 150, 16, 2, 64, 128), (BF16, 16, 150, 32, 2, 128, 64),
    (BF16, 1, 900, 2, 1, 128, 64), (F32, 1, 150, 2, 1, 64, 64), (F32, 9, 150, 16, 2, 128, 128), (F32, 16, 150, 32, 2, 64, 64)])
def test_scan_of_values_that_are_not_finite_spares_earlier_tokens(dtype, B, T, H, G, dk, dv):
    """The recurrence is causal, and the columns of x are independent: what is not finite reaches no
    earlier token of its chunk, and of x no other column.  Bits, against the same call without it."""
    k = scan_case(dtype, (B, T), H, G, dk, dv, 700 + T, B)
    d = dev(k)
    y0, s0 = gdn2.ssm_fwd(*args_of(d), d["D"], d["dt_bias"], d["s0"])
    b, h = B - 1, H - 1
    for t, value in ((0, "nan"), (5, "inf"), (17, "-inf"), (40, "nan"), (63, "inf"), (64, "nan"), (127, "inf"), (149, "nan")):
        for name in TOKENS:
            at = {"x": (b, t, h, 37), "dt": (b, t, h), "B": (b, t, G - 1, 3), "C": (b, t, G - 1, 3)}[name]
            e = dict(d)
            e[name] = d[name].clone()
            e[name][at] = float(value)
            y, s = gdn2.ssm_fwd(*args_of(e), d["D"], d["dt_bias"], d["s0"])
            assert torch.equal(y[b, :t], y0[b, :t]), (name, t)
            assert torch.equal(y[:b], y0[:b]) and torch.equal(s[:b], s0[:b]), (name, t)
            heads = H // G if name in "BC" else 1  # that read it
            assert torch.equal(y[b, :, :H - heads], y0[b, :, :H - heads]), (name, t)
            if name == "x":
                rest = torch.arange(dv, device="cuda") != 37
                assert torch.equal(y[b, :, h][:, rest], y0[b, :, h][:, rest]) and torch.equal(s[b, h][:, rest], s0[b, h][:, rest]), t
                assert not torch.isfinite(y[b, t:, h, 37]).any() and not torch.isfinite(s[b, h, :, 37]).any(), t
            elif name == "C":
                assert not torch.isfinite(y[b, t, h]).any() and torch.equal(s, s0), t
                assert torch.equal(y[b, t + 1:], y0[b, t + 1:]), t


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_packed_scan_of_padding_that_is_not_finite(dtype):
    """Padded rows taken as sequences: what lies behind a row's valid tokens, whatever it is, leaves
    them alone."""
    N, T, H, G, dk, dv = 3, 100, 2, 1, 64, 64
    valid = [1, 37, 99]
    k = scan_case(dtype, (N * T,), H, G, dk, dv, 720, N)
    d = dev(k)
    cu = torch.arange(N + 1, device="cuda") * T
    y0, _ = gdn2.ssm_fwd_varlen(*args_of(d), cu, d["D"], d["dt_bias"], d["s0"])
    for n, v in enumerate(valid):
        for m in TOKENS:
            d[m][n * T + v:(n + 1) * T] = float("nan" if n else "inf")
    y, _ = gdn2.ssm_fwd_varlen(*args_of(d), cu, d["D"], d["dt_bias"], d["s0"])
    for n, v in enumerate(valid):
        assert torch.equal(y[n * T:n * T + v], y0[n * T:n * T + v]), n
