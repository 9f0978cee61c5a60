"""spec_adjust_logits against its definition in 64 bits."""

import pytest
import torch

from paged_helpers import check_logits, logits_reference

pytestmark = pytest.mark.gpu


def rules_case(B, k, V, hist=40, seed=0, prompt=True, bias=8, mask=True, penalties=True):
    g = torch.Generator(device="cpu").manual_seed(seed)
    r = dict()
    if penalties:
        # ids outside the vocabulary are padding
        r["history"] = torch.randint(-2, V + 2, (B, hist), generator=g, dtype=torch.int32)
        r["history"][:, ::3] = torch.randint(0, min(V, 4), r["history"][:, ::3].shape, generator=g, dtype=torch.int32)
        r["hist_len"] = torch.randint(0, hist + 1, (B,), generator=g, dtype=torch.int32)
        r["prompt_len"] = torch.randint(0, hist + 1, (B,), generator=g, dtype=torch.int32) if prompt else None
        r["rep"], r["freq"], r["pres"] = 1 + torch.rand(B, generator=g), torch.rand(B, generator=g), torch.rand(B, generator=g)
    if bias:
        r["bias_tok"] = torch.randint(-1, V + 1, (B, bias), generator=g, dtype=torch.int32)
        r["bias_tok"][:, -1] = r["bias_tok"][:, 0]                     # listed twice
        r["bias_val"] = 3 * torch.randn(B, bias, generator=g)
        r["bias_len"] = torch.full((B,), bias, dtype=torch.int32)
        r["bias_len"][0] = max(1, bias // 2)
    if mask:
        words = (V + 31) // 32
        r["mask"] = torch.randint(-2 ** 31, 2 ** 31, (B, k + 1, words), generator=g, dtype=torch.int64).to(torch.int32)
        r["mask"][:, 0] = -1
        r["mask"][-1, -1] = 0                                          # nothing is allowed
    r = {n: None if t is None else t.cuda() for n, t in r.items()}
    logits = (4 * torch.randn(B, k + 1, V, generator=g)).cuda()
    drafts = torch.randint(-1, min(V, 6), (B, max(k, 1)), generator=g, dtype=torch.int32).cuda()
    return logits, drafts, r


def run(B, k, V, in_place=False, **kw):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    logits, drafts, r = rules_case(B, k, V, **kw)
    ref, mag = logits_reference(logits, drafts, V, **r)
    room = torch.full((B * (k + 1) * V + 64,), 5.0, device="cuda")
    x = room[32:32 + B * (k + 1) * V].view(B, k + 1, V)
    src = logits
    if in_place:
        x.copy_(logits)
        src = x
    bd.spec_adjust_logits(B, k, V, bd.make_logit_rules(**r), src, drafts, x)
    torch.cuda.synchronize()
    check_logits(x, ref, mag)
    assert (room[:32] == 5).all() and (room[-32:] == 5).all()


@pytest.mark.parametrize("V", [1, 2, 3, 5, 31, 33, 64, 1000, 1023, 1025, 4097, 9001])
@pytest.mark.parametrize("in_place", [False, True])
def test_vocabularies(V, in_place):
    run(3, 3, V, in_place, seed=V)


@pytest.mark.parametrize("k", [0, 1, 8])
@pytest.mark.parametrize("B", [1, 5])
def test_depths(B, k):
    run(B, k, 515, seed=k)
    run(B, k, 515, True, seed=k)


@pytest.mark.parametrize("kw", [dict(mask=False), dict(bias=0), dict(penalties=False), dict(penalties=False, bias=0),
                                dict(penalties=False, mask=False), dict(prompt=False), dict(hist=1), dict(bias=70),
                                dict(penalties=False, mask=False, bias=0)])
@pytest.mark.parametrize("in_place", [False, True])
def test_single_rules(kw, in_place):
    run(4, 2, 2050, in_place, **kw)


@pytest.mark.parametrize("B,V", [(1, 151936), (40, 30001), (600, 1003)])
def test_ranges_of_every_width(B, V):
    """Large batches and vocabularies take the wider ranges."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    logits, drafts, r = rules_case(B, 2, V, hist=300, seed=B)
    for in_place in (False, True):
        x = logits.clone()
        bd.spec_adjust_logits(B, 2, V, bd.make_logit_rules(**r), x if in_place else logits, drafts, x)
        pick = [0, B // 2, B - 1]
        sub = {n: None if t is None else t[pick] for n, t in r.items()}
        ref, mag = logits_reference(logits[pick], drafts[pick], V, **sub)
        check_logits(x[pick], ref, mag)


def test_non_finite_logits_and_lengths_past_the_array():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    logits, drafts, r = rules_case(2, 1, 300, mask=False, bias=0, seed=2)
    r["hist_len"].fill_(10 ** 6)
    r["prompt_len"].fill_(-5)
    logits[0, 0, 0] = float("-inf")
    logits[0, 0, 1] = float("inf")
    logits[0, 1, 2] = float("nan")
    out = torch.zeros_like(logits)
    bd.spec_adjust_logits(2, 1, 300, bd.make_logit_rules(**r), logits, drafts, out)
    ref, mag = logits_reference(logits, drafts, 300, **r)
    assert out[0, 0, 0] == float("-inf") and out[0, 0, 1] == float("inf") and torch.isnan(out[0, 1, 2])
    fine = torch.isfinite(logits).cpu()
    assert ((out.double().cpu() - ref).abs()[fine] <= 2.0 ** -21 * mag[fine]).all()


def test_a_graph_replays_on_new_inputs():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    logits, drafts, r = rules_case(3, 2, 2000, seed=7)
    rules, out = bd.make_logit_rules(**r), torch.zeros_like(logits)
    call = lambda: bd.spec_adjust_logits(3, 2, 2000, rules, logits, drafts, out)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    logits.mul_(-1.5)
    r["hist_len"].fill_(40)
    g.replay()
    torch.cuda.synchronize()
    ref, mag = logits_reference(logits, drafts, 2000, **r)
    check_logits(out, ref, mag)


@pytest.mark.parametrize("in_place", [False, True])
def test_more_logits_than_32_bits_count(in_place):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    B, k, V = 1010, 8, 256001 - 18000
    assert B * (k + 1) * V > 2 ** 31
    logits = torch.zeros(B, k + 1, V, device="cuda")
    logits[-1].normal_()
    _, drafts, r = rules_case(B, k, 5, hist=3, mask=False, bias=2, seed=4)
    last = logits[-1:].clone()
    out = logits if in_place else torch.empty_like(logits)
    bd.spec_adjust_logits(B, k, V, bd.make_logit_rules(**r), logits, drafts, out)
    sub = {n: None if t is None else t[-1:] for n, t in r.items()}
    ref, mag = logits_reference(last, drafts[-1:], V, **sub)
    check_logits(out[-1:], ref, mag)
