"""A paged K/V cache for the tests, and the operators' definitions in 64 bits.

Slots that no row sees hold NaN and page-table entries that no call needs hold
an id outside the pool, so that reading either shows.
"""

import math
import random

import torch


def make_case(rows, ctx, Hq, Hkv, Dh, page, seed, window=0, sinks=0, pad=0, device="cuda", spare=2):
    """Pools, table and queries of sequences with rows[b] new rows after ctx[b]
    cached positions; the pools hold every position that a row sees."""
    B = len(rows)
    g = torch.Generator(device="cpu").manual_seed(seed)
    rnd = random.Random(seed)
    total = [c + r for c, r in zip(ctx, rows)]
    width = max(1, max((t + page - 1) // page for t in total))
    need, ids = 0, []
    for t in total:
        n = (t + page - 1) // page
        ids.append(list(range(need, need + n)))
        need += n
    n_pages = need + spare
    order = list(range(n_pages))
    rnd.shuffle(order)
    table = torch.full((B, width), -7, dtype=torch.int32)
    kp = torch.full((n_pages, Hkv, page, Dh), float("nan"), dtype=torch.bfloat16)
    vp = torch.full((n_pages, Hkv, page, Dh), float("nan"), dtype=torch.bfloat16)
    seqs = []
    for b in range(B):
        n = total[b]
        k = torch.randn(n, Hkv, Dh, generator=g).to(torch.bfloat16)
        v = torch.randn(n, Hkv, Dh, generator=g).to(torch.bfloat16)
        seqs.append((k, v))
        if rows[b] == 0:
            continue
        lo = max(0, ctx[b] - window + 1) if window else 0
        for j in range(n):
            if j >= lo or j < sinks:
                pid = order[ids[b][j // page]]
                table[b, j // page] = pid
                kp[pid, :, j % page] = k[j]
                vp[pid, :, j % page] = v[j]
    start = torch.zeros(B + 1, dtype=torch.int32)
    start[1:] = torch.tensor(rows, dtype=torch.int32).cumsum(0)
    n_rows = max(1, int(start[-1]) + pad)
    q = torch.randn(n_rows, Hq, Dh, generator=g).to(torch.bfloat16)
    d = dict(B=B, Hq=Hq, Hkv=Hkv, Dh=Dh, page=page, rows=rows, ctx=ctx, window=window, sinks=sinks, n_rows=n_rows,
             seqs=seqs, q=q.to(device), k_pages=kp.to(device), v_pages=vp.to(device), table=table.to(device),
             row_start=start.to(device), ctx_len=torch.tensor(ctx, dtype=torch.int32).to(device))
    return d


def attend_reference(d, scale=None):
    """(out, lse, spread, score error) in 64 bits, rows in call order: spread is
    sum_j p_j |v_j| per output element, the score error how far an fp32 score of
    that row may be from the exact one."""
    B, Hq, Hkv, Dh = d["B"], d["Hq"], d["Hkv"], d["Dh"]
    G = Hq // Hkv
    scale = scale or 1.0 / math.sqrt(Dh)
    q = d["q"].double().cpu()
    n = q.shape[0]
    out, spread = torch.zeros(n, Hq, Dh, dtype=torch.float64), torch.zeros(n, Hq, Dh, dtype=torch.float64)
    lse, serr = torch.full((n, Hq), -math.inf, dtype=torch.float64), torch.zeros(n, Hq, dtype=torch.float64)
    r0 = 0
    for b in range(B):
        m = d["rows"][b]
        if m:
            k, v = (x.double() for x in d["seqs"][b])
            k = k.repeat_interleave(G, dim=1).permute(1, 0, 2)
            v = v.repeat_interleave(G, dim=1).permute(1, 0, 2)
            qq = q[r0:r0 + m].permute(1, 0, 2)
            s = scale * qq @ k.transpose(1, 2)
            mag = scale * qq.abs() @ k.abs().transpose(1, 2)
            pos = torch.arange(d["ctx"][b], d["ctx"][b] + m)[:, None]
            j = torch.arange(k.shape[1])[None]
            sees = j <= pos
            if d["window"]:
                sees &= (j > pos - d["window"]) | (j < d["sinks"])
            s = s.masked_fill(~sees[None], -math.inf)
            p = torch.softmax(s, dim=-1)
            out[r0:r0 + m] = (p @ v).permute(1, 0, 2)
            spread[r0:r0 + m] = (p @ v.abs()).permute(1, 0, 2)
            lse[r0:r0 + m] = torch.logsumexp(s, dim=-1).T
            # Dh products and sums in fp32, the scale, the base-2 conversion
            serr[r0:r0 + m] = mag.masked_fill(~sees[None], 0).amax(-1).T * (Dh + 4) * 2.0 ** -24
        r0 += m
    return out, lse, spread, serr


def check_attend(d, out, lse, scale=None):
    """Each weight is rounded to bf16 (2^-8) and sits under an exponential of a
    score that is off by serr and a base-2 exponential good to 2^-21; weights and
    sums are fp32; the output is rounded to bf16 (2^-8)."""
    ref, rlse, spread, serr = attend_reference(d, scale)
    n = sum(d["rows"])
    o = out[:n].double().cpu()
    e = serr[:n, :, None]
    tol = 2.0 ** -8 * ref[:n].abs() + (2.0 ** -8 + 2 * e + 2.0 ** -18) * spread[:n] * (1 + 2.0 ** -8)
    bad = (o - ref[:n]).abs() > tol
    assert torch.isfinite(o).all()
    assert not bad.any(), (float(((o - ref[:n]).abs() / tol).max()), int(bad.sum()))
    if lse is not None:
        dl = (lse[:n].double().cpu() - rlse[:n]).abs()
        tl = serr[:n] + 2.0 ** -19 + 2.0 ** -22 * rlse[:n].abs()
        assert (dl <= tl).all(), float((dl / tl).max())


def append_reference(x, pos, inv_freq, rot, half, scale):
    """Rotated rows [n, heads, Dh] in 64 bits and |x0| + |x1| of each element's pair."""
    x = x.double().cpu()
    y, mag = x.clone(), x.abs().clone()
    t = torch.arange(rot // 2)
    a, c = (t, t + rot // 2) if half else (2 * t, 2 * t + 1)
    ang = pos.double().cpu()[:, None] * inv_freq[None]
    co, si = torch.cos(ang)[:, None] * scale, torch.sin(ang)[:, None] * scale
    y[..., a] = x[..., a] * co - x[..., c] * si
    y[..., c] = x[..., c] * co + x[..., a] * si
    mag[..., a] = mag[..., c] = (x[..., a].abs() + x[..., c].abs()) * scale
    return y, mag


def logits_reference(logits, drafts, V, history=None, prompt_len=None, hist_len=None, rep=None, freq=None, pres=None,
                     bias_tok=None, bias_val=None, bias_len=None, mask=None):
    """(rules applied in 64 bits, sum of the magnitudes that met) [B, k+1, V]."""
    B, rows, _ = logits.shape
    x = logits.double().cpu().clone()
    mag = x.abs().clone()
    cpu = lambda t: None if t is None else t.cpu()  # noqa: E731
    history, prompt_len, hist_len, drafts = cpu(history), cpu(prompt_len), cpu(hist_len), cpu(drafts)
    on = rep is not None or freq is not None or pres is not None
    for b in range(B):
        for j in range(rows):
            count, seen = torch.zeros(V, dtype=torch.float64), torch.zeros(V, dtype=torch.bool)
            if on:
                if history is not None:
                    n = min(max(int(hist_len[b]), 0), history.shape[1])
                    m = min(max(int(prompt_len[b]), 0), n) if prompt_len is not None else 0
                    for i in range(n):
                        t = int(history[b, i])
                        if 0 <= t < V:
                            if i < m:
                                seen[t] = True
                            else:
                                count[t] += 1
                for i in range(j):
                    t = int(drafts[b, i])
                    if 0 <= t < V:
                        count[t] += 1
            seen |= count > 0
            r = float(rep[b]) if rep is not None else 1.0
            f = float(freq[b]) if freq is not None else 0.0
            p = float(pres[b]) if pres is not None else 0.0
            y = x[b, j]
            y = torch.where(seen, torch.where(y > 0, y / r, y * r), y)
            mag[b, j] = torch.maximum(mag[b, j], y.abs()) + abs(f) * count + abs(p) * (count > 0)
            y = y - f * count - p * (count > 0)
            if bias_tok is not None:
                for i in range(min(max(int(bias_len[b]), 0), bias_tok.shape[1])):
                    t = int(bias_tok[b, i])
                    if 0 <= t < V:
                        y[t] += float(bias_val[b, i])
                        mag[b, j, t] += abs(float(bias_val[b, i]))
            if mask is not None:
                w = mask[b, j].cpu().long() & 0xffffffff
                bits = ((w[:, None] >> torch.arange(32)) & 1).flatten()[:V].bool()
                y = torch.where(bits, y, torch.full_like(y, -math.inf))
            x[b, j] = y
    return x, mag


def check_logits(out, ref, mag):
    """At most eight fp32 roundings, each of a value no larger than the magnitudes' sum."""
    o = out.double().cpu()
    assert torch.equal(torch.isneginf(o), torch.isneginf(ref))
    fine = torch.isfinite(ref)
    assert ((o - ref).abs()[fine] <= 8 * 2.0 ** -24 * mag[fine]).all()
