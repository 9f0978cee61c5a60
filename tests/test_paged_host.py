"""Host side of the target-side operators: refusals before any device work, the
rotary tables, workspace sizes.  No GPU needed."""

import ctypes
import math
from fractions import Fraction

import pytest

from mtp_speculative_decoding_draft_gb300 import binding as bd
from mtp_speculative_decoding_draft_gb300 import build

OK_PTR = ctypes.c_void_p(1 << 20)      # aligned, never read: every call below is refused first
ODD_PTR = ctypes.c_void_p((1 << 20) + 4)
INVALID, SHAPE, WORKSPACE = -1, -2, -3


@pytest.fixture(scope="module")
def lib():
    build.build()
    return bd.library()


def cache(Hkv=8, Dh=128, page=64, n_pages=100, max_pages=10, k=OK_PTR, v=OK_PTR, t=OK_PTR):
    return bd.MtpPagedCache(Hkv, Dh, page, n_pages, max_pages, k, v, t)


def rope(turns=OK_PTR, rot=128, layout=0, scale=1.0):
    return bd.MtpRope(turns, rot, layout, scale)


def append(lib, c=None, r=None, B=2, Hq=32, n=8, rs=OK_PTR, cl=OK_PTR, q=OK_PTR, ldq=4096, k=OK_PTR, ldk=1024, v=OK_PTR,
           ldv=1024, qo=OK_PTR, ldqo=4096, ws=OK_PTR, wsb=0):
    return lib.mtp_cache_append(c or cache(), r, B, Hq, n, rs, cl, q, ldq, k, ldk, v, ldv, qo, ldqo, ws, wsb, None)


def attn(lib, c=None, B=2, Hq=32, n=8, max_rows=0, rs=OK_PTR, cl=OK_PTR, q=OK_PTR, ldq=4096, scale=0.0, window=0, sinks=0,
         out=ctypes.c_void_p(1 << 21), ldo=4096, lse=None, ws=OK_PTR, wsb=0):
    return lib.mtp_paged_attn(c or cache(), B, Hq, n, max_rows, rs, cl, q, ldq, scale, window, sinks, out, ldo, lse, ws, wsb, None)


@pytest.mark.parametrize("call", [append, attn])
def test_cache_and_row_refusals(lib, call):
    """Every argument is in order but one (a workspace of no bytes is checked last)."""
    assert call(lib) == WORKSPACE
    for c in (cache(Hkv=0), cache(n_pages=0), cache(max_pages=0), cache(k=None), cache(v=ODD_PTR), cache(t=None)):
        assert call(lib, c) == INVALID
    for c in (cache(Dh=96), cache(page=8), cache(page=48), cache(page=256), cache(n_pages=1 << 23, Hkv=8, page=128),
              cache(max_pages=1 << 25)):
        assert call(lib, c) == SHAPE
    assert call(lib, B=0) == INVALID and call(lib, n=0) == INVALID
    assert call(lib, rs=None) == INVALID and call(lib, cl=ODD_PTR) == INVALID
    assert call(lib, Hq=0) == INVALID
    assert call(lib, Hq=12) == SHAPE                          # not a multiple of Hkv
    assert call(lib, Hq=72) == SHAPE                          # groups of nine
    assert call(lib, ldq=4088) == INVALID and call(lib, ldq=4100) == INVALID
    assert call(lib, ws=None) == INVALID and call(lib, ws=ctypes.c_void_p((1 << 20) + 16)) == INVALID


def test_append_refusals(lib):
    assert append(lib, r=rope()) == WORKSPACE
    assert append(lib, q=None) == INVALID and append(lib, qo=None) == INVALID
    assert append(lib, q=None, qo=None, Hq=0) == WORKSPACE    # keys and values only
    assert append(lib, k=None) == INVALID and append(lib, ldv=1000) == INVALID
    assert append(lib, ldqo=8192) == INVALID                  # in place at another stride
    assert append(lib, r=rope(turns=None)) == INVALID
    assert append(lib, r=rope(layout=2)) == INVALID
    assert append(lib, r=rope(scale=0.0)) == INVALID and append(lib, r=rope(scale=math.nan)) == INVALID
    for rot in (0, 4, 12, 136):
        assert append(lib, r=rope(rot=rot)) == SHAPE


def test_attention_refusals(lib):
    assert attn(lib, max_rows=-1) == INVALID and attn(lib, window=-1) == INVALID and attn(lib, sinks=-1) == INVALID
    assert attn(lib, scale=-1.0) == INVALID and attn(lib, scale=math.inf) == INVALID and attn(lib, scale=math.nan) == INVALID
    assert attn(lib, q=None) == INVALID and attn(lib, out=None) == INVALID and attn(lib, out=OK_PTR) == INVALID
    assert attn(lib, n=(1 << 29) + 1) == SHAPE and append(lib, n=(1 << 29) + 1) == SHAPE
    assert attn(lib, lse=ODD_PTR) == INVALID and attn(lib, ldo=4100) == INVALID
    need = lib.mtp_paged_attn_workspace_size(2, 8, 0, 32, 8, 128)
    assert need > 256 and attn(lib, wsb=need - 1) == WORKSPACE
    for bad in ((0, 8, 0, 32, 8, 128), (2, 0, 0, 32, 8, 128), (2, 8, -1, 32, 8, 128), (2, 8, 0, 33, 8, 128), (2, 8, 0, 32, 8, 80)):
        assert lib.mtp_paged_attn_workspace_size(*bad) == 0


def test_logit_rule_refusals(lib):
    def call(B=2, k=3, V=100, rules=None, logits=OK_PTR, drafts=OK_PTR, out=OK_PTR, **kw):
        r = bd.MtpLogitRules(**kw) if rules is None else rules
        return lib.spec_adjust_logits(B, k, V, r, logits, drafts, out, None)
    assert call(B=0) == INVALID and call(k=-1) == INVALID and call(k=9) == INVALID and call(V=0) == INVALID
    assert call(logits=None) == INVALID and call(out=ODD_PTR) == INVALID and call(drafts=ODD_PTR) == INVALID
    assert lib.spec_adjust_logits(2, 3, 100, None, OK_PTR, OK_PTR, OK_PTR, None) == INVALID
    p = OK_PTR.value
    assert call(history=p) == INVALID                                        # no lengths
    assert call(history=p, hist_len=p, hist_cap=0) == INVALID
    assert call(bias_tok=p, bias_len=p, bias_cap=3) == INVALID               # no values
    assert call(bias_tok=p, bias_val=p, bias_cap=3) == INVALID
    assert call(rep=p, drafts=None) == INVALID                               # penalties need the drafts
    assert call(rep=p + 4) == INVALID and call(mask=p + 2) == INVALID
    assert call(B=1 << 20, V=1 << 30, k=0) == SHAPE


def test_binding_refusals():
    import torch
    x = torch.zeros(4, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        bd._rows(x, "q", 64)                                                     # not a CUDA tensor
    with pytest.raises(ValueError):
        bd.make_paged_cache(x, x, x)
    with pytest.raises(TypeError):
        bd.make_logit_rules(rep=torch.ones(3))


def test_turns_are_exact_to_the_last_bits(lib):
    """pos * turns mod 2^64 is the angle's fraction of a turn; against 1/(2 pi) to 60 digits."""
    import torch
    inv2pi = Fraction(159154943091895335768883763372514362034459645740456448747667, 10 ** 60)
    f = torch.tensor([1.0, 0.75, 1e-4, 10000.0 ** -0.99, 6.283185307179586, 123.456, -0.5, 1e-12, 0.0], dtype=torch.float64)
    for x, t in zip(f.tolist(), bd.rope_table(f).tolist()):
        want = Fraction(x) * inv2pi * 2 ** 64
        d = (Fraction(t) - want) % 2 ** 64
        assert min(d, 2 ** 64 - d) <= Fraction(3, 4), (x, float(d))


def test_rope_frequencies(lib):
    f, s = bd.rope_frequencies(64, 10000.0)
    assert s == 1.0 and all(abs(float(f[t]) - 10000.0 ** (-t / 32)) <= 1e-15 for t in range(32))
    g, s = bd.rope_frequencies(64, 10000.0, bd.ROPE_SCALING_LINEAR, 4.0)
    assert s == 1.0 and (g == f / 4).all()
    y, s = bd.rope_frequencies(64, 10000.0, bd.ROPE_SCALING_YARN, 8.0, 1.0, 32.0, 4096)
    assert abs(s - (0.1 * math.log(8) + 1)) < 1e-7
    for t in range(32):
        turns = 4096 * float(f[t]) / (2 * math.pi)
        keep = min(1.0, max(0.0, (turns - 1) / 31))
        assert abs(float(y[t]) - float(f[t]) * (keep + (1 - keep) / 8)) <= 1e-15
    assert y[0] == f[0] and y[-1] == f[-1] / 8
    for bad in (dict(rot_dim=0), dict(rot_dim=7), dict(rot_dim=64, base=1.0), dict(rot_dim=64, scaling=3),
                dict(rot_dim=64, scaling=1, factor=0.5), dict(rot_dim=64, scaling=2, factor=2.0, original_len=0),
                dict(rot_dim=64, scaling=2, factor=2.0, low_turns=4.0, high_turns=4.0)):
        with pytest.raises(bd.MtpError):
            bd.rope_frequencies(**bad)
    import torch
    with pytest.raises(bd.MtpError):
        bd.rope_table(torch.tensor([math.nan], dtype=torch.float64))


def test_paged_draft_refusals(lib):
    dims = bd.make_dims(2, 64, 8, 2, 64, 128, 500, 0)      # Lmax is not used
    weights = bd.MtpWeights(*[OK_PTR.value] * len(bd.WEIGHT_FIELDS))
    good = cache(Hkv=2, Dh=64)
    need = lib.mtp_paged_workspace_size(ctypes.byref(dims), 3)
    assert need > lib.mtp_workspace_size(ctypes.byref(bd.make_dims(2, 64, 8, 2, 64, 128, 500, 4)), 3)
    assert lib.mtp_paged_workspace_size(ctypes.byref(dims), 0) == 0 and lib.mtp_paged_workspace_size(None, 3) == 0

    def call(c=good, r=None, k=3, window=0, sinks=0, d=dims, wt=weights, wsb=0, ws=OK_PTR):
        draft = lib.mtp_draft_paged(d, wt, c, r, window, sinks, OK_PTR, OK_PTR, OK_PTR, k, 1.0, 0, None, OK_PTR, None, ws,
                                    wsb, None)
        step = lib.spec_step_paged(d, wt, c, r, window, sinks, OK_PTR, OK_PTR, OK_PTR, k, 1.0, 0, None, OK_PTR, None, None,
                                   OK_PTR, None, OK_PTR, OK_PTR, OK_PTR, ws, wsb, None)
        assert draft == step
        return draft
    assert call() == WORKSPACE and call(wsb=need - 1) == WORKSPACE
    assert call(r=rope(rot=64), wsb=need - 1) == WORKSPACE
    assert call(c=None) == INVALID and call(wt=None) == INVALID and call(ws=None) == INVALID and call(k=9) == INVALID
    assert call(c=cache(Hkv=8, Dh=64)) == INVALID and call(c=cache(Hkv=2, Dh=128)) == INVALID   # not the dims' heads
    assert call(c=cache(Hkv=2, Dh=64, page=40)) == SHAPE
    assert call(r=rope(rot=128)) == SHAPE and call(r=rope(rot=64, layout=7)) == INVALID
    assert call(window=-1) == INVALID and call(sinks=-1) == INVALID
    assert call(d=bd.make_dims(2, 64, 8, 3, 64, 128, 500, 0)) == SHAPE
