"""The latent-attention operators at the edges of what their arrays may hold: values
that are flagged, what the calls then leave alone, NaN and infinities."""

import pytest
import torch

from latent_helpers import attend, check_attend, check_prefill, make_latent, make_prompt, prefill

pytestmark = pytest.mark.gpu


def guarded(kind, d, **kw):
    """(out, lse, status) with the outputs and a workspace of exactly the size asked for
    inside guard bands; the workspace then serves the case as it should be."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    from mtp_speculative_decoding_draft_gb300.model import Guarded
    n, H = d["n_rows"], d["H"]
    D = d["R"] if kind == "attend" else d["Dv"]
    size = bd.latent_attn_workspace_size if kind == "attend" else bd.latent_prefill_workspace_size
    run, check = (attend, check_attend) if kind == "attend" else (prefill, check_prefill)
    guard = Guarded()
    ws = guard.alloc("workspace", size(d["B"], n, H, D), torch.uint8)
    out = guard.alloc("out", n * H * D, torch.bfloat16).view(n, H, D).fill_(7.0)
    lse = guard.alloc("lse", n * H, torch.float32).view(n, H).fill_(7.0)
    run(d, out, lse, ws, expect=None, **kw)
    guard.check()
    status = bd.get_status(ws)
    bd.clear_status(ws)
    check(d, *run(d, ws=ws))
    guard.check()
    return out, lse, status


def case(kind, rows, ctx, H=8, seed=1, **kw):
    return make_latent(rows, ctx, H, 256, 32, 32, seed, **kw) if kind == "attend" else make_prompt(rows, ctx, H, 64, 32, 64, seed, **kw)


KINDS = pytest.mark.parametrize("kind", ["attend", "prefill"])


@KINDS
@pytest.mark.parametrize("B", [4, 64, 600])
def test_row_starts_that_decrease_write_nothing(kind, B):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    rows = [1024 // B + (b < 1024 % B) for b in range(B)]
    d = case(kind, rows, [b % 70 for b in range(B)])
    back = torch.tensor([0, 1024] * (B // 2) + [0], dtype=torch.int32, device="cuda")
    out, lse, status = guarded(kind, d, row_start=back)
    assert status & bd.STATUS_BAD_ROWS
    assert (out == 7.0).all() and (lse == 7.0).all()


@KINDS
def test_row_starts_past_the_rows_are_clamped(kind):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = case(kind, [3, 90, 2], [10, 40, 0])
    past = torch.tensor([-4, 3, 93, 1 << 30], dtype=torch.int32, device="cuda")
    out, lse, status = guarded(kind, d, row_start=past)
    assert status & bd.STATUS_BAD_ROWS
    (check_attend if kind == "attend" else check_prefill)(d, out, lse)


@KINDS
@pytest.mark.parametrize("bad", [-1, 1 << 25, 2 ** 31 - 1, -2 ** 31])
def test_contexts_outside_the_cache_are_flagged(kind, bad):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = case(kind, [3, 9], [10, 40])
    if kind == "attend":
        d["pages"].nan_to_num_(0.0)
        d["table"].clamp_(min=0)
    was = d["ctx_len"].clone()
    d["ctx_len"][0] = bad
    run = attend if kind == "attend" else prefill
    out, lse = run(d, expect=bd.STATUS_BAD_CTX)
    d["ctx_len"].copy_(was)
    good, good_lse = run(d)
    assert torch.equal(out[3:], good[3:]) and torch.equal(lse[3:], good_lse[3:])      # the sequence beside it


@pytest.mark.parametrize("H", [8, 128])
def test_a_window_past_the_cache_leaves_rows_empty(H):
    """A context that the cache cannot hold: the window of its rows begins behind the last
    position, so that they see nothing."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_latent([3, 2], [10, 40], H, 256, 32, 32, seed=1, window=2)
    d["pages"].nan_to_num_(0.0)
    d["table"].clamp_(min=0)
    d["ctx_len"][0] = 1 << 20
    out, lse = attend(d, expect=bd.STATUS_BAD_CTX)
    # the context is clamped to the cache's end: row i sees what a window of two holds before it
    assert (out[1:3] == 0).all() and torch.isneginf(lse[1:3]).all()


def test_pages_outside_the_pool_are_flagged():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_latent([3, 2], [40, 80], 8, 256, 32, 32, seed=1)
    d["pages"].nan_to_num_(0.0)
    for bad in (-1, 10 ** 6):
        d["table"][0, 1] = bad
        out, _ = attend(d, expect=bd.STATUS_BAD_PAGE)
        assert torch.isfinite(out).all()


@pytest.mark.parametrize("at", [-5, 1, 1 << 30, -2 ** 31])
def test_key_starts_outside_the_keys_are_flagged(at):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_prompt([9, 20], [30, 100], 4, 64, 32, 64, seed=1)
    start = d["key_start"].clone()
    start[1] = at + (int(start[1]) if at == 1 else 0)
    out, lse = prefill(d, key_start=start, expect=bd.STATUS_BAD_CTX)
    good, good_lse = prefill(d)
    assert torch.equal(out[:9], good[:9]) and torch.equal(lse[:9], good_lse[:9])


@KINDS
def test_a_nan_in_a_query_stays_in_its_row(kind):
    d = case(kind, [40, 2], [300, 7])
    run = attend if kind == "attend" else prefill
    good, good_lse = run(d)
    d["q"][3, 1, 5] = float("nan")
    out, lse = run(d)
    hit = torch.zeros(d["n_rows"], d["H"], dtype=torch.bool, device="cuda")
    hit[3, 1] = True
    assert torch.isnan(out[hit]).all() and torch.isnan(lse[hit]).all()
    assert torch.equal(out[~hit], good[~hit]) and torch.equal(lse[~hit], good_lse[~hit])


def test_infinite_scores():
    """A score of -inf has weight zero; one of +inf leaves the row without a value."""
    d = make_prompt([40], [200], 4, 64, 32, 64, seed=2)
    d["q"].abs_()
    d["kv"][4, :, :64] = float("-inf")
    out, lse = prefill(d)
    assert torch.isfinite(out).all()
    check_prefill(d, out, lse)
    d["kv"][230, 0, :64] = float("inf")                        # rows 30 .. see it, of head 0
    out, lse = prefill(d)
    assert torch.isnan(out[30:, 0]).all() and torch.isnan(lse[30:, 0]).all()
    assert torch.isfinite(out[:30]).all() and torch.isfinite(out[:, 1:]).all()


@pytest.mark.parametrize("big", [60.0, 3000.0])
def test_scores_far_apart(big):
    """Maxima that grow along the keys by more than the accumulators are rescaled for."""
    d = make_latent([5, 30], [400, 300], 16, 256, 32, 32, seed=5)
    for b, k in enumerate(d["seqs"]):
        k *= torch.linspace(0.1, big ** 0.5, k.shape[0])[:, None]
        j = torch.arange(k.shape[0])
        d["pages"][d["table"][b, j // 32].long(), j % 32] = k.cuda()
    d["q"] *= big ** 0.5
    check_attend(d, *attend(d))


def test_refusals_of_the_binding():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    bf = dict(device="cuda", dtype=torch.bfloat16)
    pages, table = torch.zeros(4, 16, 288, **bf), torch.zeros(2, 3, device="cuda", dtype=torch.int32)
    c = bd.make_latent_cache(pages, table, 32)
    i32 = torch.zeros(8, device="cuda", dtype=torch.int32)
    rs, cl, ws = i32[:3], i32[4:6], bd.alloc_workspace(1 << 20)
    with pytest.raises(ValueError):
        bd.make_latent_cache(pages[0], table, 32)
    with pytest.raises(TypeError):
        bd.make_latent_cache(pages.float(), table, 32)
    with pytest.raises(ValueError):
        bd.mtp_latent_attn(c, rs, cl, torch.zeros(4, 2, 256, **bf), torch.zeros(4, 2, 256, **bf), None, ws, 0.1)
    with pytest.raises(ValueError):                            # more sequences than the table has
        bd.mtp_latent_attn(c, i32[:4], i32[4:7], torch.zeros(4, 2, 288, **bf), torch.zeros(4, 2, 256, **bf), None, ws, 0.1)
    with pytest.raises(bd.MtpError):                           # no scale
        bd.mtp_latent_attn(c, rs, cl, torch.zeros(4, 2, 288, **bf), torch.zeros(4, 2, 256, **bf), None, ws, 0.0)
    with pytest.raises(ValueError):
        bd.mtp_latent_append(c, None, rs, cl, torch.zeros(4, 280, **bf), None, 0.0, None, None, ws)
    with pytest.raises(ValueError):
        bd.mtp_latent_append(c, None, rs, cl, torch.zeros(4, 288, **bf), None, 0.0, torch.zeros(4, 2, 32, **bf), None, ws)
    with pytest.raises(ValueError):                            # x is not contiguous within a head
        bd.mtp_latent_heads(torch.zeros(4, 2, 64, **bf)[..., ::2], torch.zeros(2, 8, 32, **bf), torch.zeros(4, 2, 8, **bf), ws)
    with pytest.raises(ValueError):
        bd.mtp_latent_heads(torch.zeros(4, 2, 32, **bf), torch.zeros(2, 8, 40, **bf), torch.zeros(4, 2, 8, **bf), ws)
    with pytest.raises(bd.MtpError):                           # strides that are no multiple of 8
        bd.mtp_latent_heads(torch.zeros(4, 2, 36, **bf)[..., :32], torch.zeros(2, 8, 32, **bf), torch.zeros(4, 2, 8, **bf), ws)
    with pytest.raises(ValueError):
        bd.mtp_latent_expand(c, i32[:2], torch.zeros(2, 8, 32, **bf), torch.zeros(4, 2, 8, **bf), torch.zeros(4, 32, **bf), ws)
    with pytest.raises(ValueError):
        bd.mtp_latent_prefill(rs, cl, cl, torch.zeros(4, 2, 96, **bf), torch.zeros(4, 2, 120, **bf), torch.zeros(4, 32, **bf),
                              torch.zeros(4, 2, 64, **bf), None, ws, 0.1)
