"""Which sizes attention takes, on both sides of its documented bounds, without a GPU: the gradients' workspace
is more than zero bytes for sizes that are taken, and calls that are not are refused before any launch."""
import ctypes

import pytest

import gated_delta_rule_gdn2_amd as gdn2
from tests.test_abi_cpu import ERR_SHAPE, Fake
from tests.test_attention_cpu import bwd, bwd_packed, fwd, fwd_packed, lib, rot  # noqa: F401  (lib is a fixture)

LIMIT = 1 << 23  # blocks of 128 tokens of all heads


@pytest.mark.parametrize("B,T,H,G", [
    ((1 << 20) + 1, 1, 2, 1), (LIMIT - 1, 1, 1, 1), (LIMIT // 2 - 1, 1, 2, 2), (LIMIT // 7, 1, 7, 1), (LIMIT // 3, 2, 3, 3),
    (LIMIT // 5 - 4, 129, 2, 2), (63, 256, 65535, 1), (1, 128 * 128, 65535, 1), (LIMIT // 9, 1, 9, 3), (1, (1 << 29) - 1, 1, 1),
])
def test_sizes_within_the_bounds_are_taken(lib, B, T, H, G):
    """Any count of sequences and heads, however it divides into the XCDs."""
    blocks = -(-T // 128)
    if B * H * blocks >= LIMIT or B * T >= 1 << 29:
        B -= 1 + (B * H * blocks - LIMIT) // (H * blocks)
    assert B * H * blocks < LIMIT and B * T < 1 << 29
    assert gdn2.attn_bwd_workspace_bytes(B, T, T, H, G, 64) >= B * T * H * 8
    # (keys alone are bound by their key heads)
    assert gdn2.attn_bwd_workspace_bytes(B, 1, T, H, G, 64) >= B * H * 8


@pytest.mark.parametrize("N,total,H,G", [(LIMIT - 3, 200, 1, 1), (LIMIT // 7, 100, 7, 1), (LIMIT // 3 - 1, 128, 3, 3)])
def test_packed_sizes_within_the_bounds_are_taken(lib, N, total, H, G):
    assert (total // 128 + N) * H < LIMIT
    assert gdn2.attn_bwd_varlen_workspace_bytes(N, total, total, H, G, 64) >= total * H * 8


def test_sizes_behind_the_bounds_are_refused(lib):
    f = Fake()
    for kw in (dict(B=LIMIT, T=1, S=1, H=1), dict(B=LIMIT // 2, T=1, S=1, H=2), dict(B=1, T=1, S=1 << 30, H=1), dict(B=LIMIT // 4, T=1, S=513, H=1),
               dict(B=LIMIT // 4 + 1, T=129, S=1, H=2)):
        assert fwd(lib, f, **kw) == ERR_SHAPE, kw
        assert bwd(lib, f, **kw) == ERR_SHAPE, kw
        sizes = [kw[n] for n in ("B", "T", "S", "H")]
        assert gdn2.attn_bwd_workspace_bytes(*sizes, 1, 64) == 0
    for kw in (dict(N=LIMIT), dict(N=LIMIT // 2, H=2), dict(N=LIMIT - 1, T=128)):
        assert fwd_packed(lib, f, **{"H": 1, **kw}) == ERR_SHAPE, kw
    assert bwd_packed(lib, f, N=LIMIT // 2) == ERR_SHAPE


def test_more_tokens_than_rotary_takes_are_refused(lib):
    f = Fake()
    far = dict(q=ctypes.c_void_p(1 << 45), qo=ctypes.c_void_p(1 << 46))  # never read
    one = dict(far, H=1, G=0, d=2, n=2, qs=2, ks=0, qos=2, kos=0, k=None, ko=None, pos=None)
    for kw in (dict(one, tokens=1 << 27), dict(one, tokens=(1 << 31) - 1025), dict(one, tokens=1 << 27, d=192, qs=192, qos=192),
               dict(one, tokens=1 << 25, H=1024, d=64, qs=65536, qos=65536)):
        assert rot(lib, f, **kw) == ERR_SHAPE, kw
