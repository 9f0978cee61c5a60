"""Host side of the latent-attention operators: refusals before any device work,
workspace sizes.  No GPU needed."""

import ctypes
import math

import pytest

from mtp_speculative_decoding_draft_gb300 import binding as bd
from mtp_speculative_decoding_draft_gb300 import build

OK_PTR = ctypes.c_void_p(1 << 20)      # aligned, never read: every call below is refused first
OTHER = ctypes.c_void_p(1 << 21)
THIRD = ctypes.c_void_p(1 << 22)
ODD_PTR = ctypes.c_void_p((1 << 20) + 4)
INVALID, SHAPE, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bd.library()


def cache(R=512, Dr=64, page=64, n_pages=100, max_pages=10, pages=OK_PTR, t=OK_PTR):
    return bd.MtpLatentCache(R, Dr, page, n_pages, max_pages, pages, t)


def rope(turns=OK_PTR, rot=64, layout=0, scale=1.0):
    return bd.MtpRope(turns, rot, layout, scale)


def append(lib, c=None, r=None, B=2, Hq=32, n=8, rs=OK_PTR, cl=OK_PTR, kv=OK_PTR, ldkv=576, gain=OK_PTR, eps=1e-6, q=OK_PTR,
           ldq=32 * 192, hsq=192, qo=OTHER, ldqo=32 * 576, hsqo=576, ws=OK_PTR, wsb=0):
    return lib.mtp_latent_append(c or cache(), r, B, Hq, n, rs, cl, kv, ldkv, gain, eps, q, ldq, hsq, qo, ldqo, hsqo, ws, wsb, None)


def heads(lib, n=8, H=32, K=128, N=512, x=OK_PTR, ldx=32 * 192, hsx=192, w=THIRD, ldw=512, hsw=512 * 256, t=1, y=OTHER, ldy=32 * 576,
          hsy=576, ws=OK_PTR, wsb=0):
    return lib.mtp_latent_heads(n, H, K, N, x, ldx, hsx, w, ldw, hsw, t, y, ldy, hsy, ws, wsb, None)


def expand(lib, c=None, B=2, H=32, N=256, n=100, ks=OK_PTR, w=THIRD, ldw=512, hsw=512 * 256, kv=OTHER, ldkv=32 * 256, kr=OK_PTR,
           ldkr=64, ws=OK_PTR, wsb=0):
    return lib.mtp_latent_expand(c or cache(), B, H, N, n, ks, w, ldw, hsw, kv, ldkv, kr, ldkr, ws, wsb, None)


def attn(lib, c=None, B=2, Hq=32, n=8, rs=OK_PTR, cl=OK_PTR, q=OK_PTR, ldq=32 * 576, scale=0.1, window=0, sinks=0, out=OTHER,
         ldo=32 * 512, lse=None, ws=OK_PTR, wsb=0):
    return lib.mtp_latent_attn(c or cache(), B, Hq, n, rs, cl, q, ldq, scale, window, sinks, out, ldo, lse, ws, wsb, None)


def prefill(lib, B=2, H=32, Dn=128, Dr=64, Dv=128, n=8, nk=100, rs=OK_PTR, cl=OK_PTR, ks=OK_PTR, q=OK_PTR, ldq=32 * 192, kv=THIRD,
            ldkv=32 * 256, kr=OK_PTR, ldkr=64, scale=0.1, window=0, sinks=0, out=OTHER, ldo=32 * 128, lse=None, ws=OK_PTR, wsb=0):
    return lib.mtp_latent_prefill(B, H, Dn, Dr, Dv, n, nk, rs, cl, ks, q, ldq, kv, ldkv, kr, ldkr, scale, window, sinks, out, ldo,
                                  lse, ws, wsb, None)


@pytest.mark.parametrize("call", [append, expand, attn])
def test_cache_refusals(lib, call):
    """Every argument is in order but one (a workspace of no bytes is checked last)."""
    assert call(lib) == WORKSPACE
    for c in (cache(n_pages=0), cache(max_pages=0), cache(pages=None), cache(pages=ODD_PTR), cache(t=None)):
        assert call(lib, c) == INVALID
    for c in (cache(R=384), cache(R=576), cache(Dr=16), cache(Dr=128), cache(page=8), cache(page=48), cache(page=256),
              cache(n_pages=1 << 25), cache(max_pages=1 << 25)):
        assert call(lib, c) == SHAPE


@pytest.mark.parametrize("call", [append, attn, prefill])
def test_row_refusals(lib, call):
    assert call(lib, B=0) == INVALID and call(lib, n=0) == INVALID
    assert call(lib, rs=None) == INVALID and call(lib, cl=ODD_PTR) == INVALID
    assert call(lib, B=(1 << 20) + 1) == SHAPE and call(lib, n=(1 << 29) + 1) == SHAPE
    name = "H" if call is prefill else "Hq"
    assert call(lib, **{name: 0}) == INVALID and call(lib, **{name: 129}) == SHAPE


@pytest.mark.parametrize("call", [append, heads, expand, attn, prefill])
def test_workspace_refusals(lib, call):
    assert call(lib) == WORKSPACE and call(lib, wsb=255) == WORKSPACE
    assert call(lib, ws=None) == INVALID and call(lib, ws=ctypes.c_void_p((1 << 20) + 16)) == INVALID


def test_append_refusals(lib):
    assert append(lib, r=rope()) == WORKSPACE and append(lib, gain=None, eps=-1.0) == WORKSPACE
    assert append(lib, q=None, qo=None, Hq=0) == WORKSPACE                 # keys only
    assert append(lib, q=None) == INVALID and append(lib, qo=None) == INVALID
    assert append(lib, kv=None) == INVALID and append(lib, ldkv=568) == INVALID and append(lib, ldkv=580) == INVALID
    assert append(lib, gain=ODD_PTR) == INVALID
    for eps in (-1.0, math.inf, math.nan):
        assert append(lib, eps=eps) == INVALID
    assert append(lib, hsq=56) == INVALID and append(lib, hsq=196) == INVALID
    assert append(lib, ldq=31 * 192) == INVALID and append(lib, ldqo=31 * 576 + 56) == INVALID
    assert append(lib, ldq=31 * 192 + 64) == WORKSPACE                     # the last head ends the row
    assert append(lib, qo=OK_PTR) == INVALID                               # in place at other strides
    assert append(lib, qo=OK_PTR, ldqo=32 * 192, hsqo=192) == WORKSPACE
    assert append(lib, r=rope(turns=None)) == INVALID and append(lib, r=rope(layout=2)) == INVALID
    assert append(lib, r=rope(scale=0.0)) == INVALID and append(lib, r=rope(scale=math.nan)) == INVALID
    for rot in (0, 4, 12, 72):
        assert append(lib, r=rope(rot=rot)) == SHAPE
    assert append(lib, c=cache(Dr=32), ldkv=544, r=rope(rot=64)) == SHAPE
    assert append(lib, n=1 << 29, Hq=128, ldq=128 * 192, ldqo=128 * 576) == SHAPE


def test_heads_refusals(lib):
    assert heads(lib, t=0, ldw=128) == WORKSPACE
    assert heads(lib, n=0) == INVALID and heads(lib, H=0) == INVALID and heads(lib, K=0) == INVALID and heads(lib, N=-8) == INVALID
    assert heads(lib, K=4104, ldx=1 << 20, hsx=4104) == SHAPE and heads(lib, N=4104) == SHAPE and heads(lib, K=12) == SHAPE
    assert heads(lib, N=516) == SHAPE and heads(lib, H=65536) == SHAPE and heads(lib, n=(1 << 29) + 1) == SHAPE
    for p in ("x", "w", "y"):
        assert heads(lib, **{p: None}) == INVALID and heads(lib, **{p: ODD_PTR}) == INVALID
    assert heads(lib, y=OK_PTR) == INVALID and heads(lib, y=THIRD) == INVALID
    for ld in ("ldx", "hsx", "ldw", "ldy", "hsy"):
        assert heads(lib, **{ld: 8}) == INVALID and heads(lib, **{ld: 1 << 38}) == INVALID and heads(lib, **{ld: 32 * 576 + 4}) == INVALID
    assert heads(lib, hsw=0) == INVALID
    assert heads(lib, ldy=576, hsy=576) == INVALID                         # rows on top of heads
    assert heads(lib, ldy=576, hsy=8 * 576) == WORKSPACE                   # [H, rows, N]
    assert heads(lib, ldy=576, hsy=7 * 576 + 504) == INVALID
    assert heads(lib, n=1 << 29, ldy=1 << 37, hsy=512) == WORKSPACE        # heads within rows that are far apart
    assert heads(lib, n=1 << 29, ldy=1 << 30, hsy=1 << 37) == INVALID      # (no overflow in the check)


def test_expand_refusals(lib):
    assert expand(lib, B=0) == INVALID and expand(lib, H=0) == INVALID and expand(lib, n=0) == INVALID and expand(lib, N=0) == INVALID
    assert expand(lib, H=129) == SHAPE and expand(lib, N=4104, ldkv=1 << 20) == SHAPE and expand(lib, N=12) == SHAPE
    assert expand(lib, n=(1 << 29) + 1) == SHAPE
    for p in ("ks", "w", "kv", "kr"):
        assert expand(lib, **{p: None}) == INVALID and expand(lib, **{p: ODD_PTR}) == INVALID
    assert expand(lib, ldw=504) == INVALID and expand(lib, ldkv=31 * 256) == INVALID and expand(lib, ldkr=56) == INVALID
    assert expand(lib, ldkr=68) == INVALID


@pytest.mark.parametrize("call", [attn, prefill])
def test_attention_refusals(lib, call):
    assert call(lib, window=-1) == INVALID and call(lib, sinks=-1) == INVALID
    for scale in (0.0, -1.0, math.inf, math.nan):
        assert call(lib, scale=scale) == INVALID
    assert call(lib, q=None) == INVALID and call(lib, out=None) == INVALID and call(lib, out=OK_PTR) == INVALID
    assert call(lib, lse=ODD_PTR) == INVALID
    assert call(lib, ldq=31 * 192) == INVALID and call(lib, ldo=8) == INVALID and call(lib, ldo=(1 << 20) + 4) == INVALID


def test_prefill_refusals(lib):
    for k in ({"Dn": 96}, {"Dv": 256}, {"Dr": 16}, {"Dr": 128}, {"nk": (1 << 30) + 1}):
        assert prefill(lib, **k) == SHAPE
    assert prefill(lib, nk=0) == INVALID and prefill(lib, ks=None) == INVALID and prefill(lib, kv=ODD_PTR) == INVALID
    assert prefill(lib, kr=None) == INVALID and prefill(lib, ldkv=31 * 256) == INVALID and prefill(lib, ldkr=32) == INVALID


def test_workspace_sizes(lib):
    attn_size, pre_size = lib.mtp_latent_attn_workspace_size, lib.mtp_latent_prefill_workspace_size
    for bad in ((0, 8, 32, 512), (2, 0, 32, 512), (2, 8, 0, 512), (2, 8, 129, 512), (2, 8, 32, 384), ((1 << 20) + 1, 8, 32, 512),
                (2, (1 << 29) + 1, 32, 512)):
        assert attn_size(*bad) == 0
    for bad in ((0, 8, 32, 128), (2, 0, 32, 128), (2, 8, 129, 128), (2, 8, 32, 96)):
        assert pre_size(*bad) == 0
    for H in (1, 16, 40, 128):                                             # on either side of the choice of kernels
        for n in (2, 9, 64, 5000):
            need = attn_size(2, n, H, 512)
            assert need > 256 and attn(lib, Hq=H, n=n, ldq=H * 576, ldo=H * 512, wsb=need - 1) == WORKSPACE
            need = pre_size(2, n, H, 128)
            assert need > 256 and prefill(lib, H=H, n=n, ldq=H * 192, ldkv=H * 256, ldo=H * 128, wsb=need - 1) == WORKSPACE
    # a list of items that 31 bits do not count is refused
    assert attn_size(1 << 20, 1 << 29, 128, 512) == 0 or attn_size(1 << 20, 1 << 29, 128, 512) > 1 << 30
    assert attn(lib, B=1 << 20, n=1 << 29, Hq=128, ldq=128 * 576, ldo=128 * 512) in (SHAPE, WORKSPACE)
