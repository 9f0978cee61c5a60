"""The target-side operators at the edges of what their arrays may hold: values that
are flagged, and what the calls then leave alone."""

import pytest
import torch

from paged_helpers import check_attend, make_case

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
