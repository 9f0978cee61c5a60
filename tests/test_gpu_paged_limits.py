"""The target-side operators at the edges of what their arrays may hold: values that
are flagged, and what the calls then leave alone."""

import pytest
import torch

from paged_helpers import attend_reference, check_attend, make_case

pytestmark = pytest.mark.gpu


def guarded_attention(d, max_rows, row_start):
    """(out, lse, status) with out, lse and a workspace of exactly the size asked for
    inside guard bands."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    from mtp_speculative_decoding_draft_gb300.model import Guarded
    n, Hq, Hkv, Dh = d["n_rows"], d["Hq"], d["Hkv"], d["Dh"]
    guard = Guarded()
    ws = guard.alloc("workspace", bd.paged_attn_workspace_size(d["B"], n, max_rows, Hq, Hkv, Dh), torch.uint8)
    out = guard.alloc("out", n * Hq * Dh, torch.bfloat16).view(n, Hq, Dh).fill_(7.0)
    lse = guard.alloc("lse", n * Hq, torch.float32).view(n, Hq).fill_(7.0)
    cache = bd.make_paged_cache(d["k_pages"], d["v_pages"], d["table"])
    bd.mtp_paged_attn(cache, row_start, d["ctx_len"], d["q"], out, lse, ws, window=d["window"], sinks=d["sinks"],
                      max_rows=max_rows)
    torch.cuda.synchronize()
    guard.check()
    status = bd.get_status(ws)
    bd.clear_status(ws)
    # the same workspace serves a call that is in order
    bd.mtp_paged_attn(cache, d["row_start"], d["ctx_len"], d["q"], x := torch.zeros_like(d["q"]), y := torch.zeros_like(lse), ws,
                      window=d["window"], sinks=d["sinks"], max_rows=max_rows)
    torch.cuda.synchronize()
    guard.check()
    assert bd.get_status(ws) == 0
    check_attend(d, x, y)
    return out, lse, status


@pytest.mark.parametrize("max_rows", [0, 2])                   # the tensor-core kernel, the streaming kernel
@pytest.mark.parametrize("B", [4, 64, 600])                    # more sequences than the plan has threads, too
def test_row_starts_that_decrease_write_nothing(B, max_rows):
    """Rows counted again and again would fill more of the plan than the workspace has."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    rows = [1024 // B + (b < 1024 % B) for b in range(B)]
    d = make_case(rows, [b % 70 for b in range(B)], 16, 8, 64, 32, seed=B)
    back = torch.tensor([0, 1024] * (B // 2) + [0], dtype=torch.int32, device="cuda")
    out, lse, status = guarded_attention(d, max_rows, back)
    assert status & bd.STATUS_BAD_ROWS
    assert (out == 7.0).all() and (lse == 7.0).all()


@pytest.mark.parametrize("max_rows", [0, 2])
def test_row_starts_past_the_rows_are_clamped(max_rows):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_case([3, 90, 2], [10, 40, 0], 16, 8, 64, 32, seed=1)
    past = torch.tensor([-4, 3, 93, 1 << 30], dtype=torch.int32, device="cuda")
    d["k_pages"].nan_to_num_(0.0)
    d["v_pages"].nan_to_num_(0.0)
    out, lse, status = guarded_attention(d, max_rows, past)
    assert status & bd.STATUS_BAD_ROWS
    check_attend(d, out, lse)                                  # clamped to the rows that there are


# A context that no position can have: the row is not written, the sequences beside it are.
@pytest.mark.parametrize("bad", [-1, -3, 2 ** 31 - 1, 2 ** 31 - 2, -2 ** 31])
@pytest.mark.parametrize("B", [3, 40])                         # row starts from a lane each, and by search
def test_an_append_at_no_position_writes_nothing(bad, B):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_case([2] * B, [5 + b for b in range(B)], 4, 2, 64, 16, seed=B)
    n = d["n_rows"]
    g = torch.Generator(device="cuda").manual_seed(1)
    k, v = (torch.randn(n, 2, 64, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    was = [d[name].clone() for name in ("k_pages", "v_pages")]
    d["ctx_len"][1] = bad
    ws = bd.alloc_workspace(256)
    bd.mtp_cache_append(bd.make_paged_cache(d["k_pages"], d["v_pages"], d["table"]), None, d["row_start"], d["ctx_len"], None,
                        k, v, None, ws)
    torch.cuda.synchronize()
    assert bd.get_status(ws) == bd.STATUS_BAD_CTX
    for b in range(B):
        if b != 1:
            for i in range(2):
                for pool, x in zip(was, (k, v)):
                    pool[int(d["table"][b, (5 + b + i) // 16]), :, (5 + b + i) % 16] = x[2 * b + i]
    for name, pool in zip(("k_pages", "v_pages"), was):
        assert torch.equal(d[name].view(torch.int16), pool.view(torch.int16))


# The draft's depths are appended one by one behind ctx_len: none of them lands on a
# position that a wrapped or clamped sum gives.
@pytest.mark.parametrize("bad", [-1, -2, 2 ** 31 - 1, 2 ** 31 - 2])
def test_a_paged_draft_at_no_position_writes_nothing(bad):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    from mtp_speculative_decoding_draft_gb300 import workloads as W
    from test_gpu_paged_draft import MID, paged_module
    w, wts, ctx = MID, W.make_weights(MID), W.make_context(MID)
    m, _ = paged_module(w, ctx, wts, 64)
    for pool in m.cache.tensors[:2]:
        pool.nan_to_num_(0.0)
    was = [pool.clone() for pool in m.cache.tensors[:2]]
    m.ctx_len.fill_(bad)
    m.draft_paged(w.T, 0)
    torch.cuda.synchronize()
    assert m.status() & bd.STATUS_BAD_CTX
    m.check_canaries()
    for pool, x in zip(m.cache.tensors[:2], was):
        assert torch.equal(pool.view(torch.int16), x.view(torch.int16))


def attended(d, max_rows):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    n, Hq = d["n_rows"], d["Hq"]
    out, lse = torch.zeros_like(d["q"]), torch.zeros(n, Hq, device="cuda")
    ws = bd.alloc_workspace(bd.paged_attn_workspace_size(d["B"], n, max_rows, Hq, d["Hkv"], d["Dh"]))
    bd.mtp_paged_attn(bd.make_paged_cache(d["k_pages"], d["v_pages"], d["table"]), d["row_start"], d["ctx_len"], d["q"], out, lse,
                      ws, max_rows=max_rows)
    torch.cuda.synchronize()
    assert bd.get_status(ws) == 0
    return out, lse


@pytest.mark.parametrize("ctx", [20, 3000])                    # one share, and states that are joined
@pytest.mark.parametrize("Dh,max_rows", [(32, 0), (64, 0), (128, 0), (64, 3), (128, 3)])
def test_a_nan_in_sight_is_a_nan_in_lse(Dh, max_rows, ctx):
    """A NaN score leaves the row's sum without a value: lse says so, as the output
    does, and not that the row saw no key.  Every other row keeps its value."""
    d = make_case([40, 2], [ctx, 7], 8, 2, Dh, 32, seed=Dh)
    good, good_lse = attended(d, max_rows)
    check_attend(d, good, good_lse)
    # query head 1 of row 3; the key at position ctx + 30, which rows 30 .. 39 of kv head 1 see
    clean = d["q"].clone()
    d["q"][3, 1, 5] = float("nan")
    pos = ctx + 30
    d["k_pages"][int(d["table"][0, pos // 32]), 1, pos % 32, 9] = float("nan")
    out, lse = attended(d, max_rows)
    hit = torch.zeros(d["n_rows"], 8, dtype=torch.bool, device="cuda")
    hit[3, 1] = True
    hit[30:40, 4:] = True
    assert torch.isnan(lse[hit]).all() and torch.isnan(out[hit]).all()
    # the rest within the definition's bounds (a row's maximum may move with its warp's)
    check_attend(dict(d, q=clean), torch.where(hit[..., None], good, out), torch.where(hit, good_lse, lse))


@pytest.mark.parametrize("max_rows", [0, 3])
def test_infinite_scores(max_rows):
    """A key of score +inf: weight inf / inf, no value.  One of -inf: weight zero."""
    d = make_case([40], [200], 4, 1, 64, 32, seed=2)
    good, good_lse = attended(d, max_rows)
    q = d["q"]
    q.abs_()
    d["k_pages"][int(d["table"][0, 0]), 0, 4, :] = float("-inf")
    out, lse = attended(d, max_rows)
    k, v = d["seqs"][0]
    k[4] = float("-inf")
    assert torch.isfinite(out).all()
    s = (q.double().cpu().permute(1, 0, 2) @ k.double().permute(1, 2, 0)) / 8
    s = s.masked_fill(torch.arange(240)[None, None] > torch.arange(200, 240)[None, :, None], float("-inf"))
    ref = torch.logsumexp(s, dim=-1).T
    # the score's fp32 products, as in check_attend, of |q| |k| below 64 * 5 * 5 / 8
    assert ((lse.double().cpu() - ref).abs() <= 200 * 68 * 2.0 ** -24 + 2.0 ** -19 + 2.0 ** -22 * ref.abs()).all()
    d["k_pages"][int(d["table"][0, 0]), 0, 4, :] = float("inf")
    out, lse = attended(d, max_rows)
    assert torch.isnan(out).all() and torch.isnan(lse).all()


@pytest.mark.parametrize("B", [513, 600, 1024, 1025, 1100])
@pytest.mark.parametrize("Hq,Hkv,Dh", [(4, 2, 64), (8, 1, 128)])
def test_large_batches_on_the_tensor_cores(B, Hq, Hkv, Dh):
    """More sequences than the plan's one block has threads, and than it keeps the
    blocks of in shared memory; empty ones first, last and between; two chunks."""
    rows = [(b * 7) % 4 for b in range(B)]
    ctx = [(b * 37) % 91 for b in range(B)]
    rows[0] = rows[1] = rows[-1] = rows[-2] = 0
    rows[B // 2], rows[min(B - 3, 512)] = 150, 90
    d = make_case(rows, ctx, Hq, Hkv, Dh, 16, seed=B, pad=3)
    out, lse = attended(d, 0)
    check_attend(d, out, lse)
    n = sum(rows)
    assert (out[n:] == 0).all() and (lse[n:] == 0).all()


@pytest.mark.parametrize("Hq,Hkv,Dh,rows", [(32, 8, 128, 4), (8, 1, 64, 2), (10, 2, 128, 3), (4, 2, 32, 8), (8, 8, 64, 1)])
@pytest.mark.parametrize("ctx,window", [(40, 0), (1000, 0), (9000, 0), (2000, 300)])
def test_few_rows_carry_their_weights_in_16_bits(Hq, Hkv, Dh, rows, ctx, window):
    """Up to 16 packed rows: a weight is a bf16 value and a second one that holds what the
    first rounding left, at most 2^-8 of it; the second's own rounding is 2^-8 of that."""
    d = make_case([rows, 1], [ctx, ctx // 3], Hq, Hkv, Dh, 32, seed=ctx + Dh, window=window, sinks=3 if window else 0)
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    out = torch.zeros_like(d["q"])
    ws = bd.alloc_workspace(bd.paged_attn_workspace_size(2, d["n_rows"], rows, Hq, Hkv, Dh))
    bd.mtp_paged_attn(bd.make_paged_cache(d["k_pages"], d["v_pages"], d["table"]), d["row_start"], d["ctx_len"], d["q"], out, None,
                      ws, window=window, sinks=d["sinks"], max_rows=rows)
    torch.cuda.synchronize()
    assert bd.get_status(ws) == 0
    ref, _, spread, serr = attend_reference(d)
    # the weights' two roundings, scores, exponentials (2^-21) and fp32 sums as in
    # check_attend, and the output's own rounding (2^-8)
    tol = 2.0 ** -8 * ref.abs() + (2.0 ** -16 + 2 * serr[..., None] + 2.0 ** -18) * spread * (1 + 2.0 ** -8)
    err = (out.double().cpu() - ref).abs()
    assert (err <= tol).all(), float((err / tol).max())
