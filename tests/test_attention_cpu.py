"""The attention block's argument checks, without a GPU: the C ABI's (host addresses that are never
dereferenced: every call here is refused, or has nothing to do, before any launch) and the binding's."""
import ctypes
import math
import os

import pytest
import torch

import gated_delta_rule_gdn2_amd as gdn2
from tests.test_abi_cpu import BF16, ERR_ALIAS, ERR_MISALIGNED, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_WORKSPACE, F32, OK, Fake

INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(gdn2.library_path()):
        pytest.skip("libgdn2.so not built")
    return gdn2._load()


def args_of(f, names, over):
    a = {n: f.p(i) for i, n in enumerate(names.split())}
    a.update(over)
    return a.values()


def fwd(lib, f, B=1, T=64, S=64, H=2, G=1, d=64, qs=None, ks=None, vs=None, window=0, scale=0.125, dtype=BF16, ws=None, wb=0, **over):
    return lib.gdn2_attn_fwd(*args_of(f, "q k v o lse", over), B, T, S, H, G, d, H * d if qs is None else qs,
                             G * d if ks is None else ks, G * d if vs is None else vs, window, scale, dtype, ws, wb, None)


def fwd_packed(lib, f, N=2, T=64, S=64, H=2, G=1, d=64, window=0, scale=0.125, dtype=BF16, ws=None, wb=0, **over):
    return lib.gdn2_attn_fwd_varlen(*args_of(f, "q k v o lse cu cuk", over), N, T, S, H, G, d, H * d, G * d, G * d, window, scale,
                                    dtype, ws, wb, None)


def bwd(lib, f, B=1, T=64, S=64, H=2, G=1, d=64, qs=None, ks=None, vs=None, window=0, scale=0.125, dtype=BF16, ws="own", wb=1 << 16,
        **over):
    return lib.gdn2_attn_bwd(*args_of(f, "do q k v o lse dq dk dv", over), B, T, S, H, G, d, H * d if qs is None else qs,
                             G * d if ks is None else ks, G * d if vs is None else vs, window, scale, dtype,
                             f.p(10) if ws == "own" else ws, wb, None)


def bwd_packed(lib, f, N=2, T=64, S=64, ws="own", wb=1 << 16, **over):
    return lib.gdn2_attn_bwd_varlen(*args_of(f, "do q k v o lse dq dk dv cu cuk", over), N, T, S, 2, 1, 64, 128, 64, 64, 0, 0.125,
                                    BF16, f.p(11) if ws == "own" else ws, wb, None)


def step(lib, f, N=3, H=2, G=1, d=64, C=16, qs=None, ks=None, vs=None, window=0, scale=0.125, dtype=BF16, ws=None, wb=0, **over):
    return lib.gdn2_attn_step(*args_of(f, "q k v kc vc pos o", over), N, H, G, d, C, H * d if qs is None else qs,
                              G * d if ks is None else ks, G * d if vs is None else vs, window, scale, dtype, ws, wb, None)


def rot(lib, f, tokens=8, T=8, H=2, G=1, d=64, n=64, qs=128, ks=64, qos=128, kos=64, scale=1.0, dtype=BF16, **over):
    return lib.gdn2_rotary(*args_of(f, "q k freq pos qo ko", over), tokens, T, H, G, d, n, qs, ks, qos, kos, 0, 0, scale, dtype, None)


def rms(lib, f, rows=4, width=64, eps=1e-6, dtype=BF16, rdt=BF16, **over):
    return lib.gdn2_rms_norm(*args_of(f, "x r gamma y h rstd", over), rows, width, eps, dtype, rdt, None)


def rms8(lib, f, rows=4, width=64, eps=1e-6, dtype=BF16, rdt=BF16, **over):
    return lib.gdn2_rms_norm_fp8(*args_of(f, "x r gamma y s h rstd", over), rows, width, eps, dtype, rdt, None)


def rms_bwd(lib, f, rows=4, width=64, dtype=BF16, rdt=BF16, wb=0, ws=None, **over):
    return lib.gdn2_rms_norm_bwd(*args_of(f, "dy h gamma rstd dh dx dgamma", over), ws, wb, rows, width, dtype, rdt, None)


def test_attention_refusals(lib):
    f = Fake()
    for call, names in ((fwd, "q k v o"), (bwd, "do q k v o lse dq dk dv")):
        for n in names.split():
            assert call(lib, f, **{n: None}) == ERR_NULL, (call, n)
        for kw in (dict(B=0), dict(T=-1), dict(S=-1), dict(H=0), dict(G=0), dict(H=3, G=2), dict(qs=120), dict(ks=56), dict(vs=56),
                   dict(qs=1 << 22), dict(ks=1 << 22), dict(vs=1 << 22), dict(H=1 << 16), dict(B=1 << 40), dict(B=1 << 31),
                   dict(T=1 << 31), dict(S=(1 << 31) - 1024), dict(B=1 << 24, H=2), dict(B=1 << 20, T=1 << 20), dict(window=-1),
                   dict(scale=0.0), dict(scale=-1.0), dict(scale=NAN), dict(scale=INF)):
            assert call(lib, f, **kw) == ERR_SHAPE, (call, kw)
        for kw in (dict(d=96), dict(d=256), dict(dtype=3)):
            assert call(lib, f, **kw) == ERR_UNSUPPORTED, (call, kw)
        for kw in (dict(q=f.p(0, 8)), dict(k=f.p(1, 2)), dict(v=f.p(2, 4)), dict(o=f.p(3, 8)), dict(lse=f.p(4, 2)), dict(qs=132),
                   dict(ks=68), dict(vs=65)):
            assert call(lib, f, **kw) == ERR_MISALIGNED, (call, kw)
    for kw in (dict(o=f.p(0)), dict(o=f.p(1, 64)), dict(lse=f.p(2)), dict(o=f.p(4)), dict(lse=f.p(3, 16)), dict(o=f.p(0, 63 * 512), qs=256)):
        assert fwd(lib, f, **kw) == ERR_ALIAS, kw
    for kw in (dict(dq=f.p(1)), dict(dk=f.p(0)), dict(dv=f.p(5)), dict(dq=f.p(4)), dict(dk=f.p(3)), dict(dk=f.p(8)), dict(dq=f.p(7, -16)),
               dict(ws=f.p(2)), dict(ws=f.p(8))):
        assert bwd(lib, f, **kw) == ERR_ALIAS, kw
    assert fwd(lib, f, T=0, q=None, o=None) == OK  # no queries: nothing to do
    assert bwd(lib, f, T=0, S=0) == OK


def test_packed_refusals(lib):
    f = Fake()
    for n in "q k v o cu cuk".split():
        assert fwd_packed(lib, f, **{n: None}) == ERR_NULL, n
    for n in "do q k v o lse dq dk dv cu cuk".split():
        assert bwd_packed(lib, f, **{n: None}) == ERR_NULL, n
    for kw in (dict(N=0), dict(N=1 << 31), dict(T=-1), dict(N=1 << 23)):
        assert fwd_packed(lib, f, **kw) == ERR_SHAPE, kw
        assert bwd_packed(lib, f, **kw) == ERR_SHAPE, kw
    assert fwd_packed(lib, f, cu=f.p(5, 4)) == ERR_MISALIGNED
    assert bwd_packed(lib, f, cuk=f.p(10, 4)) == ERR_MISALIGNED
    for kw in (dict(o=f.p(5)), dict(lse=f.p(6))):
        assert fwd_packed(lib, f, **kw) == ERR_ALIAS, kw
    for kw in (dict(dq=f.p(9)), dict(dv=f.p(10)), dict(ws=f.p(9))):
        assert bwd_packed(lib, f, **kw) == ERR_ALIAS, kw


def test_workspaces(lib):
    f = Fake()
    a16 = lambda slot, off=0: ctypes.c_void_p((f.p(slot).value + 15) // 16 * 16 + off)
    # whole where the blocks of queries fill the GPU, and where there are few keys
    assert gdn2.attn_fwd_workspace_bytes(8, 4096, 4096, 16, 8, 128) == 0
    assert gdn2.attn_fwd_workspace_bytes(1, 4, 200, 2, 1, 64) == 0
    assert gdn2.attn_fwd_workspace_bytes(1, 4, 100000, 2, 1, 64, window=100) == 0
    assert gdn2.attn_fwd_workspace_bytes(0, 4, 4, 2, 1, 64) == 0 and gdn2.attn_fwd_workspace_bytes(1, 4, 4, 2, 1, 96) == 0
    assert fwd(lib, f, ws=a16(8), wb=1 << 18) == ERR_WORKSPACE
    assert fwd(lib, f, wb=1) == ERR_WORKSPACE
    need = gdn2.attn_fwd_workspace_bytes(1, 4, 4096, 2, 1, 64)
    assert need > 0 and need % 4 == 0
    long = dict(T=4, S=4096)
    assert fwd(lib, f, ws=a16(8), wb=need - 1, **long) == ERR_WORKSPACE
    assert fwd(lib, f, ws=None, wb=need, **long) == ERR_WORKSPACE
    assert fwd(lib, f, ws=a16(8, 8), wb=need, **long) == ERR_MISALIGNED
    for slot in range(5):
        assert fwd(lib, f, ws=a16(slot), wb=need, **long) == ERR_ALIAS, slot
    need = gdn2.attn_fwd_varlen_workspace_bytes(2, 8, 4096, 2, 1, 64)
    assert need > 0
    assert fwd_packed(lib, f, T=8, S=4096, ws=a16(8), wb=need - 4) == ERR_WORKSPACE
    assert fwd_packed(lib, f, T=8, S=4096, ws=a16(6), wb=need) == ERR_ALIAS
    # gradients: eight bytes a query and head, more where heads share keys and workgroups are few
    assert gdn2.attn_bwd_workspace_bytes(1, 100, 100, 6, 6, 64) == 4800 and gdn2.attn_bwd_workspace_bytes(1, 0, 4, 6, 6, 64) == 0
    assert gdn2.attn_bwd_varlen_workspace_bytes(2, 100, 100, 6, 6, 64) == 4800
    parts = gdn2.attn_bwd_workspace_bytes(1, 4096, 4096, 4, 1, 64) - 4096 * 4 * 8
    assert parts > 0 and parts % (2 * 4096 * 64 * 4) == 0
    assert bwd(lib, f, ws=None, wb=0) == ERR_WORKSPACE and bwd(lib, f, wb=64 * 2 * 8 - 1) == ERR_WORKSPACE
    assert bwd(lib, f, ws=f.p(10, 8)) == ERR_MISALIGNED
    # steps
    assert gdn2.attn_step_workspace_bytes(3, 2, 1, 64, 16) == 0 and gdn2.attn_step_workspace_bytes(3, 3, 2, 64, 4096) == 0
    need = gdn2.attn_step_workspace_bytes(3, 2, 1, 64, 4096)
    assert need > 0 and gdn2.attn_step_workspace_bytes(3, 2, 1, 64, 4096, window=100) == 0
    assert step(lib, f, ws=a16(8), wb=1 << 18) == ERR_WORKSPACE
    for ws, wb, kw, want in ((a16(8), need - 1, {}, ERR_WORKSPACE), (a16(8, 4), need, {}, ERR_MISALIGNED), (a16(6), need, {}, ERR_ALIAS),
                             (a16(3), need, {}, ERR_ALIAS), (a16(5), need, {}, ERR_ALIAS)):
        assert step(lib, f, C=4096, ws=ws, wb=wb, **kw) == want
    # norms: none for few rows
    assert gdn2.rms_norm_bwd_workspace_bytes(3, 64) == 0 and gdn2.rms_norm_bwd_workspace_bytes(4, 0) == 0
    need = gdn2.rms_norm_bwd_workspace_bytes(4096, 64)
    assert need > 0
    assert rms_bwd(lib, f, rows=4096) == ERR_WORKSPACE
    assert rms_bwd(lib, f, rows=4096, ws=f.p(8), wb=need - 1) == ERR_WORKSPACE
    assert rms_bwd(lib, f, rows=4096, ws=f.p(8, 8), wb=need) == ERR_MISALIGNED
    assert rms_bwd(lib, f, rows=4096, ws=f.p(5), wb=need) == ERR_ALIAS


def test_step_refusals(lib):
    f = Fake()
    for n in "q k v kc vc pos o".split():
        assert step(lib, f, **{n: None}) == ERR_NULL, n
    for kw in (dict(N=0), dict(H=0), dict(G=0), dict(C=0), dict(H=3, G=2), dict(qs=64), dict(ks=56), dict(vs=8), dict(qs=1 << 31),
               dict(ks=1 << 31), dict(vs=1 << 31), dict(N=1 << 23), dict(C=1 << 31), dict(window=-1), dict(scale=0.0), dict(scale=NAN),
               dict(H=1 << 16)):
        assert step(lib, f, **kw) == ERR_SHAPE, kw
    for kw in (dict(d=32), dict(dtype=2)):
        assert step(lib, f, **kw) == ERR_UNSUPPORTED, kw
    for kw in (dict(q=f.p(0, 8)), dict(k=f.p(1, 2)), dict(v=f.p(2, 4)), dict(kc=f.p(3, 8)), dict(vc=f.p(4, 8)), dict(pos=f.p(5, 4)),
               dict(o=f.p(6, 8)), dict(qs=132), dict(ks=68), dict(vs=66)):
        assert step(lib, f, **kw) == ERR_MISALIGNED, kw
    for kw in (dict(o=f.p(0)), dict(kc=f.p(1)), dict(vc=f.p(3, 16)), dict(kc=f.p(5)), dict(o=f.p(4))):
        assert step(lib, f, **kw) == ERR_ALIAS, kw


def test_rotary_refusals(lib):
    f = Fake()
    for n in "q k freq qo ko".split():
        assert rot(lib, f, **{n: None}) == ERR_NULL, n
    for kw in (dict(tokens=-1), dict(tokens=1 << 31), dict(T=0), dict(H=0), dict(G=-1), dict(d=0, n=0), dict(d=514, n=64, qs=1028, ks=514, qos=1028, kos=514),
               dict(n=0), dict(n=3), dict(n=66), dict(qs=127), dict(ks=63), dict(qos=100), dict(kos=8), dict(qs=1 << 31),
               dict(kos=1 << 31), dict(H=1 << 16, qs=1 << 30, qos=1 << 30), dict(scale=0.0), dict(scale=NAN), dict(scale=INF)):
        assert rot(lib, f, **kw) == ERR_SHAPE, kw
    assert rot(lib, f, dtype=2) == ERR_UNSUPPORTED
    for kw in (dict(q=f.p(0, 1)), dict(ko=f.p(5, 1)), dict(freq=f.p(2, 2)), dict(pos=f.p(3, 4)), dict(k=f.p(1, 2), dtype=F32)):
        assert rot(lib, f, **kw) == ERR_MISALIGNED, kw
    # in place is for the same address and stride; parts of one tensor share no byte
    for kw in (dict(qo=f.p(0, 2)), dict(qo=f.p(0), qos=136), dict(ko=f.p(0)), dict(qo=f.p(1)), dict(ko=f.p(4)), dict(qo=f.p(2)),
               dict(ko=f.p(3)), dict(qo=f.p(0, 128), qs=256, qos=256), dict(ko=f.p(0, 128), ks=256, kos=256, qs=256, qos=256)):
        assert rot(lib, f, **kw) == ERR_ALIAS, kw
    assert rot(lib, f, tokens=0) == OK


def test_rms_refusals(lib):
    f = Fake()
    for n in "x gamma y h r".split():
        assert rms(lib, f, **{n: None}) == ERR_NULL, n
        assert rms8(lib, f, **{n: None}) == ERR_NULL, n
    assert rms8(lib, f, s=None) == ERR_NULL
    for n in "dy h gamma rstd dx dgamma".split():
        assert rms_bwd(lib, f, **{n: None}) == ERR_NULL, n
    for kw in (dict(rows=-1), dict(rows=1 << 31), dict(width=0), dict(width=16385)):
        for call in (rms, rms8, rms_bwd):
            assert call(lib, f, **kw) == ERR_SHAPE, (call, kw)
    for eps in (-1e-6, NAN, INF):
        assert rms(lib, f, eps=eps) == ERR_SHAPE and rms8(lib, f, eps=eps) == ERR_SHAPE
    for kw in (dict(dtype=2), dict(dtype=F32, rdt=BF16), dict(rdt=2)):
        for call in (rms, rms8, rms_bwd):
            assert call(lib, f, **kw) == ERR_UNSUPPORTED, (call, kw)
    for kw in (dict(x=f.p(0, 8)), dict(r=f.p(1, 8)), dict(gamma=f.p(2, 4)), dict(y=f.p(3, 8)), dict(h=f.p(4, 2)), dict(rstd=f.p(5, 2))):
        assert rms(lib, f, **kw) == ERR_MISALIGNED, kw
    for kw in (dict(dy=f.p(0, 8)), dict(h=f.p(1, 8)), dict(dh=f.p(4, 8)), dict(dx=f.p(5, 8)), dict(dgamma=f.p(6, 4)), dict(rstd=f.p(3, 2))):
        assert rms_bwd(lib, f, **kw) == ERR_MISALIGNED, kw
    for kw in (dict(y=f.p(0)), dict(y=f.p(1)), dict(h=f.p(0)), dict(h=f.p(1, 16)), dict(rstd=f.p(3)), dict(y=f.p(4)), dict(h=f.p(2))):
        assert rms(lib, f, **kw) == ERR_ALIAS, kw
    for kw in (dict(s=f.p(3)), dict(s=f.p(6)), dict(y=f.p(5))):
        assert rms8(lib, f, **kw) == ERR_ALIAS, kw
    for kw in (dict(dx=f.p(0)), dict(dx=f.p(1)), dict(dgamma=f.p(2)), dict(dx=f.p(4, 16)), dict(dgamma=f.p(4)), dict(dx=f.p(6))):
        assert rms_bwd(lib, f, **kw) == ERR_ALIAS, kw
    assert rms(lib, f, rows=0) == OK and rms8(lib, f, rows=0, s=None) == OK


def test_supported():
    for dtype in (torch.bfloat16, torch.float32):
        assert gdn2.supported("attn", 64, 64, dtype) and gdn2.supported("attn", 128, 128, dtype)
        assert not gdn2.supported("attn", 64, 128, dtype) and not gdn2.supported("attn", 96, 96, dtype)


def test_binding_refuses_cpu_tensors():
    z = torch.zeros
    q, k = z(1, 4, 2, 64), z(1, 4, 1, 64)
    for call in (lambda: gdn2.attn_fwd(q, k, k), lambda: gdn2.attn_fwd_varlen(q[0], k[0], k[0], z(2, dtype=torch.int64)),
                 lambda: gdn2.attn_bwd(q, q, k, k, q, z(1, 4, 2)), lambda: gdn2.rotary(q, k, z(8)), lambda: gdn2.rms_norm(q, z(64)),
                 lambda: gdn2.attn_step(q[0], k[0], k[0], z(4, 8, 1, 64), z(4, 8, 1, 64), z(4, dtype=torch.int64)),
                 lambda: gdn2.rms_norm_fp8(q, z(64)), lambda: gdn2.rms_norm_bwd(q, q, z(64), z(1, 4, 2))):
        with pytest.raises(ValueError, match="runs on the GPU"):
            call()
    with pytest.raises(ValueError, match="q must be|x must be"):
        gdn2.attn_fwd(q[0], k[0], k[0])


def test_rotary_frequencies():
    f = gdn2.rotary_frequencies(8)
    assert f.dtype == torch.float32 and f.tolist() == pytest.approx([1.0, 0.1, 0.01, 0.001], rel=1e-7)
    assert torch.equal(gdn2.rotary_frequencies(64, 500.0, factor=4.0), (500.0 ** (-torch.arange(0, 64, 2).double() / 64) / 4).float())
    # by turns in the context learned: the fast ones stay, the slow ones are divided, a line between
    length = 4096
    f, g = gdn2.rotary_frequencies(128).double(), gdn2.rotary_frequencies(128, factor=8.0, length=length, low=2.0, high=16.0).double()
    turns = length * f / (2 * math.pi)
    assert torch.equal(g[turns > 16.01], f[turns > 16.01])
    assert torch.allclose(g[turns < 1.99], f[turns < 1.99] / 8, rtol=1e-6)
    mid = (turns > 2) & (turns < 16)
    share = (turns[mid] - 2) / 14
    assert mid.any() and torch.allclose(g[mid], f[mid] * (share + (1 - share) / 8), rtol=1e-6)
    for kw in (dict(rot=7), dict(rot=0), dict(rot=8, factor=0.0), dict(rot=8, factor=2.0, length=0), dict(rot=8, factor=2.0, length=10, low=3.0, high=3.0)):
        with pytest.raises(ValueError):
            gdn2.rotary_frequencies(**kw)
