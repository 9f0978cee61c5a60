"""The target's side of two speculative steps in a row, as a serving program runs
them: append the candidates' keys and values, attend them over the pages, put the
rules on the head's logits, verify, advance the contexts by what was accepted."""

import pytest
import torch

from mtp_speculative_decoding_draft_gb300.model import Verifier
from paged_helpers import append_reference, check_attend, check_logits, logits_reference

pytestmark = pytest.mark.gpu

B, k, V, Hq, Hkv, Dh, page = 5, 3, 1203, 8, 2, 64, 16


@pytest.mark.parametrize("captured", [False, True])
def test_two_steps(captured):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    g = torch.Generator(device="cuda").manual_seed(5)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    ctx = [0, 13, 16, 45, 100]
    width = (max(ctx) + 2 * (k + 1) + page - 1) // page
    table = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width).contiguous()
    pools = [torch.full((B * width, Hkv, page, Dh), float("nan"), device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    seqs = []
    for b in range(B):
        kv = [rnd(ctx[b], Hkv, Dh).to(torch.bfloat16) for _ in range(2)]
        for pool, x in zip(pools, kv):
            for j in range(ctx[b]):
                pool[int(table[b, j // page]), :, j % page] = x[j]
        seqs.append([x.cpu() for x in kv])
    cache = bd.make_paged_cache(pools[0], pools[1], table)
    freq, _ = bd.rope_frequencies(Dh)
    rope = bd.make_rope(bd.rope_table(freq).cuda(), Dh)
    n = B * (k + 1)
    row_start = torch.arange(0, n + 1, k + 1, device="cuda", dtype=torch.int32)
    ctx_len = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    qkv, head = rnd(n, (Hq + 2 * Hkv) * Dh).to(torch.bfloat16), 0.2 * rnd(Hq * Dh, V)
    q, key, val = (x.view(n, -1, Dh) for x in qkv.split([Hq * Dh, Hkv * Dh, Hkv * Dh], dim=1))
    q_rot, out = torch.zeros(n, Hq, Dh, device="cuda", dtype=torch.bfloat16), torch.zeros(n, Hq, Dh, device="cuda", dtype=torch.bfloat16)
    lse, logits = torch.zeros(n, Hq, device="cuda"), torch.zeros(B, k + 1, V, device="cuda")
    drafts = torch.randint(0, V, (B, k), generator=g, device="cuda", dtype=torch.int32)
    history = torch.randint(0, 30, (B, 64), generator=g, device="cuda", dtype=torch.int32)
    mask = torch.full((B, k + 1, (V + 31) // 32), -1, device="cuda", dtype=torch.int32)
    mask[1, 0] = 0x0f0f0f0f
    r = dict(history=history, prompt_len=torch.full((B,), 9, device="cuda", dtype=torch.int32),
             hist_len=torch.full((B,), 20, device="cuda", dtype=torch.int32), rep=1.1 + 0 * rnd(B).abs(),
             freq=0.3 + 0 * rnd(B), pres=0.2 + 0 * rnd(B), mask=mask)
    rules = bd.make_logit_rules(**r)
    raw = torch.zeros_like(logits)
    ws, ws_a = bd.alloc_workspace(256), bd.alloc_workspace(bd.paged_attn_workspace_size(B, n, k + 1, Hq, Hkv, Dh))
    v = Verifier(B, k, V)

    def step():
        bd.mtp_cache_append(cache, rope, row_start, ctx_len, q, key, val, q_rot, ws)
        bd.mtp_paged_attn(cache, row_start, ctx_len, q_rot, out, lse, ws_a, max_rows=k + 1)
        torch.mm(out.view(n, -1).float(), head, out=raw.view(n, V))
        logits.copy_(raw)
        bd.spec_adjust_logits(B, k, V, rules, logits, drafts, logits)
        v(1.0, 0, logits, None, drafts)

    run = step
    if captured:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            step()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
        run = graph.replay

    for turn in range(2):
        if turn:
            qkv.copy_(rnd(*qkv.shape).to(torch.bfloat16))
        # a sequence whose drafts are what the target says, the others' are random
        run()
        torch.cuda.synchronize()
        drafts[0].copy_(logits[0].argmax(-1)[:k].to(torch.int32))
        run()
        torch.cuda.synchronize()
        assert bd.get_status(ws) == 0 and bd.get_status(ws_a) == 0
        # keys and queries rotated, the pages hold them behind the context
        pos = torch.cat([torch.arange(c, c + k + 1) for c in ctx])
        for got, x in ((q_rot, q), (None, key)):
            ref, mag = append_reference(x, pos, freq, Dh, True, 1.0)
            if got is None:
                seq = torch.arange(B).repeat_interleave(k + 1)
                got = pools[0].cpu()[table.cpu()[seq, pos // page].long(), :, pos % page]
            assert ((got.double().cpu() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -20 * mag).all()
            new_keys = got
        now = [[torch.cat([s[0], new_keys[b * (k + 1):(b + 1) * (k + 1)]]), torch.cat([s[1], val[b * (k + 1):(b + 1) * (k + 1)].cpu()])]
               for b, s in enumerate(seqs)]
        check_attend(dict(B=B, Hq=Hq, Hkv=Hkv, Dh=Dh, rows=[k + 1] * B, ctx=ctx, window=0, sinks=0, q=q_rot, seqs=now), out, lse)
        ref, mag = logits_reference(raw, drafts, V, **r)
        check_logits(logits, ref, mag)
        toks, length, acc = v.results()
        best = logits.argmax(-1).cpu().tolist()
        for b in range(B):
            a = 0
            while a < k and int(drafts[b, a]) == best[b][a]:
                a += 1
            assert acc[b] == a and length[b] == a + 1 and toks[b][a] == best[b][a]
        if turn == 0:
            # accepted rows stay, rejected ones are overwritten by the next append
            ctx = [c + int(a) for c, a in zip(ctx, length)]
            seqs = [[x[:c] for x in s] for s, c in zip(now, ctx)]
            ctx_len.copy_(torch.tensor(ctx, dtype=torch.int32))
            for b in range(B):
                history[b, 20:20 + int(length[b])] = torch.from_numpy(toks[b][:length[b]]).cuda()
                r["hist_len"][b] = 20 + int(length[b])
    assert len({int(x) for x in ctx_len}) > 1
