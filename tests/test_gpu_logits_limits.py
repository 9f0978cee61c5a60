"""spec_adjust_logits where a copy does not land: the rows that it misses come by
plain loads, and nothing of the shared memory that was never filled reaches the
output.  The stall is a copy that is not issued: no fault and no endless wait."""

import time

import pytest
import torch

from paged_helpers import check_logits, logits_reference
from test_gpu_logits import rules_case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("V,kw", [(9001, dict()), (4096, dict(mask=False)), (2, dict(bias=0))])
def test_a_copy_that_never_lands_changes_no_logit(V, kw):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    B, k = 2, 4
    logits, drafts, r = rules_case(B, k, V, seed=V, **kw)
    ref, mag = logits_reference(logits, drafts, V, **r)
    room = torch.full((B * (k + 1) * V + 64,), 5.0, device="cuda")
    out = room[32:-32].view(B, k + 1, V)
    rules = bd.make_logit_rules(**r)
    torch.cuda.synchronize()
    t0 = time.perf_counter()
    bd.selftest_logits_wait(B, k, V, rules, logits, drafts, out)
    torch.cuda.synchronize()
    dt = time.perf_counter() - t0
    assert 1.9 < dt < 30.0, "the waits gave up after %.2f s (limit 2 s, and as long again before the exit)" % dt
    check_logits(out, ref, mag)
    assert (room[:32] == 5).all() and (room[-32:] == 5).all()
    # and the context is as usable as before
    out.zero_()
    bd.spec_adjust_logits(B, k, V, rules, logits, drafts, out)
    torch.cuda.synchronize()
    check_logits(out, ref, mag)


@pytest.mark.parametrize("V", [30004, 30001])
@pytest.mark.parametrize("kw", [dict(), dict(penalties=False, bias=0), dict(bias=70, hist=300)])
def test_nine_rows_of_one_block_under_a_mask(V, kw):
    """Enough ranges that a block takes all rows of its range: the ring of rows in shared
    memory goes round four times and a half, with the rows on 16-byte boundaries or not."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    B, k = 24, 8
    assert B * ((V + 2047) // 2048) >= 2 * torch.cuda.get_device_properties(0).multi_processor_count
    logits, drafts, r = rules_case(B, k, V, seed=V, **kw)
    out = torch.zeros_like(logits)
    bd.spec_adjust_logits(B, k, V, bd.make_logit_rules(**r), logits, drafts, out)
    torch.cuda.synchronize()
    pick = [0, 11, B - 1]
    sub = {n: None if t is None else t[pick] for n, t in r.items()}
    ref, mag = logits_reference(logits[pick], drafts[pick], V, **sub)
    check_logits(out[pick], ref, mag)
    # the rules in place, on the same rows
    bd.spec_adjust_logits(B, k, V, bd.make_logit_rules(**r), logits, drafts, logits)
    assert torch.equal(logits, out)
