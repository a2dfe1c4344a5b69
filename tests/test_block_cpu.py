"""The state space block's argument checks, without a GPU: the C ABI's (host addresses that are never
dereferenced: every call here is refused, or has nothing to do, before any HIP call) and the binding's."""
import ctypes
import os

import pytest
import torch

import gated_delta_rule_gdn2_amd as gdn2
from tests.test_abi_cpu import BF16, ERR_ALIAS, ERR_MISALIGNED, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_WORKSPACE, F32, OK, Fake


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn2.library_path()):
        pytest.skip("libgdn2.so not built")
    return gdn2._load()


def ssm(lib, f, B=1, T=64, H=2, G=1, dk=64, dv=64, xs=None, ts=None, bs=None, cs=None, dtype=BF16, ws=None, wb=0, **over):
    a = {n: f.p(i) for i, n in enumerate("x dt b c A D bias s0 y sT".split())}
    a.update(over)
    return lib.gdn2_ssm_fwd(*a.values(), B, T, H, G, dk, dv, H * dv if xs is None else xs, H if ts is None else ts,
                            G * dk if bs is None else bs, G * dk if cs is None else cs, dtype, 1, ws, wb, None)


def packed(lib, f, N=2, total=64, H=2, G=1, dk=64, dv=64, dtype=BF16, ws=None, wb=0, **over):
    a = {n: f.p(i) for i, n in enumerate("x dt b c A D bias s0 y sT cu".split())}
    a.update(over)
    return lib.gdn2_ssm_fwd_varlen(*a.values(), N, total, H, G, dk, dv, H * dv, H, G * dk, G * dk, dtype, 1, ws, wb, None)


def step(lib, f, N=3, H=2, G=1, dk=64, dv=64, dtype=BF16, **over):
    a = {n: f.p(i) for i, n in enumerate("x dt b c A D bias s y".split())}
    a.update(over)
    return lib.gdn2_ssm_step(*a.values(), N, H, G, dk, dv, H * dv, H, G * dk, G * dk, dtype, 1, None)


def test_scan_refusals(lib):
    f = Fake()
    for n in "x dt b c A y".split():
        assert ssm(lib, f, **{n: None}) == ERR_NULL, n
    for kw in (dict(B=0), dict(T=0), dict(H=0), dict(G=0), dict(H=3, G=2), dict(xs=120), dict(ts=1), dict(bs=56),
               dict(cs=8), dict(xs=1 << 22), dict(ts=1 << 22), dict(H=1 << 16), dict(B=1 << 40, T=1 << 40),
               dict(B=1 << 30, H=8)):
        assert ssm(lib, f, **kw) == ERR_SHAPE, kw
    for kw in (dict(dk=96), dict(dv=32), dict(dtype=3)):
        assert ssm(lib, f, **kw) == ERR_UNSUPPORTED, kw
    for kw in (dict(x=f.p(0, 8)), dict(b=f.p(2, 2)), dict(c=f.p(3, 4)), dict(y=f.p(8, 8)), dict(s0=f.p(7, 4)),
               dict(A=f.p(4, 2)), dict(dt=f.p(1, 1)), dict(xs=132), dict(bs=68), dict(cs=65)):
        assert ssm(lib, f, **kw) == ERR_MISALIGNED, kw
    for kw in (dict(y=f.p(0)), dict(y=f.p(1)), dict(sT=f.p(2, 16)), dict(y=f.p(7)), dict(sT=f.p(8)),
               dict(sT=f.p(7, 64)), dict(sT=f.p(4)), dict(y=f.p(0, 64 * 200 * 2), xs=256)):
        assert ssm(lib, f, **kw) == ERR_ALIAS, kw


def test_scan_workspace_refusals(lib):
    f = Fake(nbytes=1 << 24, slots=12)
    assert lib.gdn2_ssm_fwd_workspace_bytes(0, 64, 2, 64, 64, BF16) == 0
    assert lib.gdn2_ssm_fwd_workspace_bytes(1, 64, 2, 96, 64, BF16) == 0
    assert lib.gdn2_ssm_fwd_workspace_bytes(1, 64, 2, 64, 64, BF16) == 0  # one chunk: nothing to cut
    assert ssm(lib, f, ws=f.p(10), wb=1 << 20) == ERR_WORKSPACE
    assert ssm(lib, f, wb=1) == ERR_WORKSPACE
    # packed: a workspace where total_T is more than a segment
    assert lib.gdn2_ssm_fwd_varlen_workspace_bytes(2, 64, 2, 64, 64, BF16) == 0
    assert packed(lib, f, ws=f.p(11), wb=1 << 20) == ERR_WORKSPACE
    need = lib.gdn2_ssm_fwd_varlen_workspace_bytes(2, 4096, 2, 64, 64, BF16)
    assert need > 0 and need == gdn2.ssm_fwd_varlen_workspace_bytes(2, 4096, 2, 64, 64)
    a256 = lambda slot: f.p(slot, -f.p(slot).value % 256)
    assert packed(lib, f, total=4096, ws=a256(11), wb=need - 1) == ERR_WORKSPACE
    assert packed(lib, f, total=4096, ws=None, wb=need) == ERR_WORKSPACE
    assert packed(lib, f, total=4096, ws=ctypes.c_void_p(a256(11).value + 16), wb=need) == ERR_MISALIGNED
    for slot in (0, 1, 2, 3, 7, 8, 9):
        assert packed(lib, f, total=4096, ws=a256(slot), wb=need) == ERR_ALIAS, slot
    need = lib.gdn2_ssm_fwd_workspace_bytes(1, 8192, 2, 64, 64, BF16)
    assert need > 0
    assert ssm(lib, f, T=8192, ws=a256(8), wb=need) == ERR_ALIAS
    assert ssm(lib, f, T=8192, ws=a256(10), wb=need - 1) == ERR_WORKSPACE


def test_scan_limits(lib):
    """Sizes whose indexes or whose launch would pass 32 bits (a tensor expanded along its tokens
    takes no memory for them)."""
    f = Fake()
    top = (1 << 31) - 1024
    assert ssm(lib, f, T=top) == ERR_SHAPE and packed(lib, f, total=top) == ERR_SHAPE
    assert lib.gdn2_ssm_fwd_workspace_bytes(1, top, 2, 64, 64, BF16) == 0
    assert lib.gdn2_ssm_fwd_varlen_workspace_bytes(2, top, 2, 64, 64, BF16) == 0
    assert ssm(lib, f, B=1 << 23, T=1, H=1) == ERR_SHAPE and packed(lib, f, N=1 << 22, H=2) == ERR_SHAPE
    assert step(lib, f, N=1 << 22, H=2) == ERR_SHAPE


def test_conv_limits(lib):
    """Launches of 2^32 threads: 2^21 sequences of one token of 8192 channels (34 GB) are one."""
    f = Fake()
    assert conv(lib, f, B=1 << 21, T=1, C=8192) == ERR_SHAPE
    assert conv(lib, f, B=1, T=1 << 24, C=16384) == ERR_SHAPE
    a = [f.p(i) for i in range(7)]
    assert lib.gdn2_short_conv_varlen(*a, 1 << 21, 64, 8192, 8192, BF16, None) == ERR_SHAPE
    assert lib.gdn2_short_conv_step(a[0], a[1], a[2], a[5], a[4], 1 << 21, 8192, 8192, BF16, None) == ERR_SHAPE


def test_packed_and_step_refusals(lib):
    f = Fake()
    assert packed(lib, f, cu=None) == ERR_NULL
    assert packed(lib, f, x=None) == ERR_NULL
    assert packed(lib, f, N=0) == ERR_SHAPE and packed(lib, f, total=-1) == ERR_SHAPE
    assert packed(lib, f, cu=f.p(10, 4)) == ERR_MISALIGNED
    assert packed(lib, f, y=f.p(10)) == ERR_ALIAS and packed(lib, f, sT=f.p(10)) == ERR_ALIAS
    assert packed(lib, f, total=0, x=None, dt=None, b=None, c=None, y=None, sT=None) == OK
    for n in "x dt b c A s y".split():
        assert step(lib, f, **{n: None}) == ERR_NULL, n
    assert step(lib, f, N=0) == ERR_SHAPE and step(lib, f, H=3, G=2) == ERR_SHAPE
    assert step(lib, f, dk=32) == ERR_UNSUPPORTED
    assert step(lib, f, s=f.p(7, 8)) == ERR_MISALIGNED
    assert step(lib, f, s=f.p(0)) == ERR_ALIAS and step(lib, f, y=f.p(7, 64)) == ERR_ALIAS


def conv(lib, f, B=2, T=5, C=64, xs=None, dtype=BF16, **over):
    a = {n: f.p(i) for i, n in enumerate("x taps bias s0 y sT".split())}
    a.update(over)
    return lib.gdn2_short_conv(*a.values(), B, T, C, C if xs is None else xs, dtype, None)


def test_conv_refusals(lib):
    f = Fake()
    for n in ("x", "taps", "y"):
        assert conv(lib, f, **{n: None}) == ERR_NULL, n
    for kw in (dict(B=0), dict(T=0), dict(C=0), dict(C=12), dict(xs=56), dict(xs=1 << 22), dict(C=1 << 22, xs=1 << 22),
               dict(B=1 << 31, T=1)):
        assert conv(lib, f, **kw) == ERR_SHAPE, kw
    assert conv(lib, f, dtype=2) == ERR_UNSUPPORTED
    for kw in (dict(x=f.p(0, 1)), dict(taps=f.p(1, 4)), dict(bias=f.p(2, 4)), dict(sT=f.p(5, 2))):
        assert conv(lib, f, **kw) == ERR_MISALIGNED, kw
    for kw in (dict(y=f.p(0)), dict(sT=f.p(0, 64)), dict(y=f.p(3)), dict(sT=f.p(3, 128)), dict(sT=f.p(4)), dict(y=f.p(1))):
        assert conv(lib, f, **kw) == ERR_ALIAS, kw
    a = [f.p(i) for i in range(6)]
    call = lambda cu, N=2, total=9, y=a[4]: lib.gdn2_short_conv_varlen(*a[:4], y, a[5], cu, N, total, 64, 64, BF16, None)
    assert call(None) == ERR_NULL and call(f.p(6), N=0) == ERR_SHAPE and call(f.p(6), total=-1) == ERR_SHAPE
    assert call(f.p(6, 4)) == ERR_MISALIGNED and call(f.p(4, 8)) == ERR_ALIAS and call(f.p(6), y=None) == ERR_NULL
    assert lib.gdn2_short_conv_varlen(None, a[1], None, None, None, None, f.p(6), 2, 0, 64, 64, BF16, None) == OK
    st = lambda s, y=a[4]: lib.gdn2_short_conv_step(a[0], a[1], a[2], s, y, 2, 64, 64, BF16, None)
    assert st(None) == ERR_NULL and st(a[0]) == ERR_ALIAS and st(f.p(5, 8)) == ERR_MISALIGNED and st(a[5], None) == ERR_NULL


def norm(lib, f, rows=4, width=100, eps=1e-5, dtype=F32, **over):
    a = {n: f.p(i) for i, n in enumerate("x gamma beta y mean rstd".split())}
    a.update(over)
    return lib.gdn2_layer_norm(*a.values(), rows, width, eps, dtype, None)


def norm_bwd(lib, f, rows=400, width=100, dtype=F32, wb=None, **over):
    a = {n: f.p(i) for i, n in enumerate("dy x gamma mean rstd dx dgamma dbeta ws".split())}
    a.update(over)
    if wb is None:
        wb = lib.gdn2_layer_norm_bwd_workspace_bytes(rows, width)
    return lib.gdn2_layer_norm_bwd(*a.values(), wb, rows, width, dtype, None)


def test_norm_refusals(lib):
    f = Fake()
    for n in ("x", "gamma", "y", "mean", "rstd"):  # one statistic without the other
        assert norm(lib, f, **{n: None}) == ERR_NULL, n
    for kw in (dict(rows=-1), dict(width=0), dict(width=16385), dict(eps=-1.0), dict(eps=float("nan")), dict(rows=1 << 31)):
        assert norm(lib, f, **kw) == ERR_SHAPE, kw
    assert norm(lib, f, dtype=4) == ERR_UNSUPPORTED
    for kw in (dict(x=f.p(0, 4)), dict(mean=f.p(4, 2)), dict(beta=f.p(2, 8))):
        assert norm(lib, f, **kw) == ERR_MISALIGNED, kw
    for kw in (dict(y=f.p(0)), dict(mean=f.p(1)), dict(rstd=f.p(4)), dict(rstd=f.p(3, 16))):
        assert norm(lib, f, **kw) == ERR_ALIAS, kw
    assert norm(lib, f, rows=0, x=None, y=None) == OK
    for n in ("dy", "x", "gamma", "mean", "rstd", "dx", "dgamma"):
        assert norm_bwd(lib, f, **{n: None}) == ERR_NULL, n
    assert norm_bwd(lib, f, rows=-1) == ERR_SHAPE and norm_bwd(lib, f, width=20000) == ERR_SHAPE
    assert norm_bwd(lib, f, ws=None) == ERR_WORKSPACE
    assert norm_bwd(lib, f, wb=lib.gdn2_layer_norm_bwd_workspace_bytes(400, 100) - 1) == ERR_WORKSPACE
    assert norm_bwd(lib, f, ws=f.p(8, 8)) == ERR_MISALIGNED and norm_bwd(lib, f, dx=f.p(5, 4)) == ERR_MISALIGNED
    for kw in (dict(dx=f.p(0)), dict(dgamma=f.p(2)), dict(dbeta=f.p(6)), dict(ws=f.p(1)), dict(ws=f.p(7))):
        assert norm_bwd(lib, f, **kw) == ERR_ALIAS, kw
    assert lib.gdn2_layer_norm_bwd_workspace_bytes(4, 20000) == 0
    assert lib.gdn2_layer_norm_bwd_workspace_bytes(4, 100) == 0 < lib.gdn2_layer_norm_bwd_workspace_bytes(400, 100)


def test_binding_refuses_cpu_tensors_and_odd_layouts():
    x = torch.zeros(2, 5, 3, 64)
    with pytest.raises(ValueError, match="GPU"):
        gdn2.ssm_fwd(x, x[..., 0], x, x, x[0, 0, :, 0])
    with pytest.raises(ValueError, match="GPU"):
        gdn2.short_conv(x[:, :, 0], torch.zeros(64, 4))
    with pytest.raises(ValueError, match="GPU"):
        gdn2.layer_norm(x, torch.ones(64))
    with pytest.raises(TypeError):
        gdn2.layer_norm(x.double().cuda() if torch.cuda.is_available() else _on_gpu_double(x), torch.ones(64))


def _on_gpu_double(x):
    class Double(torch.Tensor):
        is_cuda = True
    return x.double().as_subclass(Double)


def test_token_strides():
    """The binding's reading of strides: a token's own elements contiguous, one stride between tokens."""
    t, cpu = gdn2.block._tokens, torch.device("cpu")
    wide = torch.zeros(2, 5, 3 * 64 + 40)
    read = lambda v, inner: t("x", v, tuple(v.shape), inner, torch.float32, cpu)
    assert read(wide[..., :192].unflatten(-1, (3, 64)), 2) == 232
    assert read(wide[..., 192:], 1) == 232
    assert read(wide[:, :1, :192], 1) == 5 * 232      # one token of each sequence
    assert read(wide[:1, :1, :192], 1) == 192         # a single token
    assert read(wide[:1, :, 8:16], 1) == 232
    assert read(torch.zeros(0, 3, 64), 2) == 192
    assert read(wide.transpose(0, 1).contiguous().transpose(0, 1)[:, :1], 1) == 232
    for bad in (wide[:, :4, :192], wide[..., ::2], wide.transpose(0, 1), wide[..., :192].unflatten(-1, (64, 3)).transpose(2, 3),
                wide[:1, :1].expand(2, 5, 232)):
        with pytest.raises(ValueError):
            read(bad, 2 if bad.dim() == 4 else 1)
    with pytest.raises(ValueError):
        t("x", wide, (2, 5, 100), 1, torch.float32, cpu)
    with pytest.raises(TypeError):
        t("x", wide, tuple(wide.shape), 1, torch.bfloat16, cpu)
