"""A latent cache for the tests, and the latent operators' definitions in 64 bits.

Slots that no row sees hold NaN and page-table entries that no call needs hold
an id outside the pool, so that reading either shows.
"""

import math
import random

import torch


def make_latent(rows, ctx, H, R, Dr, page, seed, window=0, sinks=0, pad=0, spare=2, device="cuda"):
    """Pool, table and queries of sequences with rows[b] new rows after ctx[b] cached
    positions; the pool holds every position that a row sees."""
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
    pages = torch.full((n_pages, page, R + Dr), float("nan"), dtype=torch.bfloat16)
    seqs = []
    for b in range(B):
        n = total[b]
        k = torch.randn(n, R + Dr, generator=g).to(torch.bfloat16)
        seqs.append(k)
        if rows[b] == 0 or n == 0:
            continue
        lo = max(0, ctx[b] - window + 1) if window else 0
        j = torch.arange(n)
        j = j[(j >= lo) | (j < sinks)]
        pid = torch.tensor([order[i] for i in ids[b]])[j // page]
        table[b, j // page] = pid.to(torch.int32)
        pages[pid, j % page] = k[j]
    start = torch.zeros(B + 1, dtype=torch.int32)
    start[1:] = torch.tensor(rows, dtype=torch.int32).cumsum(0)
    n_rows = max(1, int(start[-1]) + pad)
    q = torch.randn(n_rows, H, R + Dr, generator=g).to(torch.bfloat16)
    return dict(B=B, H=H, R=R, Dr=Dr, page=page, rows=rows, ctx=ctx, window=window, sinks=sinks, n_rows=n_rows, seqs=seqs,
                scale=(R + Dr) ** -0.5, q=q.to(device), pages=pages.to(device), table=table.to(device),
                row_start=start.to(device), ctx_len=torch.tensor(ctx, dtype=torch.int32).to(device))


def sees(ctx, n, keys, window, sinks):
    pos, j = torch.arange(ctx, ctx + n)[:, None], torch.arange(keys)[None]
    s = j <= pos
    if window:
        s &= (j > pos - window) | (j < sinks)
    return s


def attention(q, k, v, visible, scale, device="cpu"):
    """One sequence in 64 bits: q [n, H, D], k [L, H or 1, D], v [L, H or 1, Dv].  Returns
    (out, lse, spread, score error): spread is sum_j p_j |v_j|, the score error how far an
    fp32 score of the row may be from the exact one."""
    q, k, v = (x.to(device).double().transpose(0, 1) for x in (q, k, v))
    s = scale * (q @ k.transpose(1, 2)).masked_fill(~visible[None], -math.inf)
    mag = scale * (q.abs() @ k.abs().transpose(1, 2)).masked_fill(~visible[None], 0)
    lse = torch.logsumexp(s, dim=-1)
    p = torch.where(torch.isinf(lse)[..., None], torch.zeros_like(s), (s - lse[..., None]).exp())
    # D products and sums in fp32, which the tensor cores may cut off instead of rounding
    # (2^-23), the scale, the base-2 conversion
    err = mag.amax(-1) * (q.shape[-1] + 4) * 2.0 ** -23
    return (p @ v).transpose(0, 1), lse.t(), (p @ v.abs()).transpose(0, 1), err.t()


def attend_reference(d):
    n, H, R = d["n_rows"], d["H"], d["R"]
    out, spread = torch.zeros(n, H, R, dtype=torch.float64), torch.zeros(n, H, R, dtype=torch.float64)
    lse, err = torch.full((n, H), -math.inf, dtype=torch.float64), torch.zeros(n, H, dtype=torch.float64)
    r = 0
    for b, m in enumerate(d["rows"]):
        if m:
            k = d["seqs"][b]
            e = slice(r, r + m)
            out[e], lse[e], spread[e], err[e] = attention(d["q"][e], k[:, None], k[:, None, :R],
                                                          sees(d["ctx"][b], m, k.shape[0], d["window"], d["sinks"]), d["scale"])
        r += m
    return out, lse, spread, err


def check_rows(ref, out, lse, n, keys):
    """ref: (out, lse, spread, score error).  A weight is rounded to bf16 (2^-8) and sits
    under an exponential of a score that is off by err, good to 2^-21; fp32 sums of at most
    `keys` terms, cut off or rounded (2^-23 each), in the weights' sum and in the product;
    the output is rounded to bf16 (2^-8)."""
    want, wlse, spread, err = (x[:n] for x in ref)
    o, sums = out[:n].double().cpu(), (2 * keys + 64) * 2.0 ** -23
    tol = 2.0 ** -8 * want.abs() + (2.0 ** -8 + 2 * err[..., None] + 2.0 ** -18 + sums) * spread * (1 + 2.0 ** -8)
    bad = (o - want).abs() > tol
    assert torch.isfinite(o).all()
    assert not bad.any(), (float(((o - want).abs() / tol.clamp(min=1e-30)).max()), int(bad.sum()))
    if lse is not None:
        z = lse[:n].double().cpu()
        assert torch.equal(torch.isneginf(z), torch.isneginf(wlse))
        fine = torch.isfinite(wlse)
        tl = err + 2.0 ** -19 + sums + 2.0 ** -22 * wlse.abs()
        assert ((z - wlse).abs()[fine] <= tl[fine]).all(), float(((z - wlse).abs() / tl)[fine].max())


def check_attend(d, out, lse):
    check_rows(attend_reference(d), out, lse, sum(d["rows"]), max(c + r for c, r in zip(d["ctx"], d["rows"])))


def attend(d, out=None, lse=None, ws=None, row_start=None, expect=0):
    """mtp_latent_attn of the case; (out, lse)."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    n, H, R = d["n_rows"], d["H"], d["R"]
    out = torch.full((n, H, R), 7.0, device="cuda", dtype=torch.bfloat16) if out is None else out
    lse = torch.full((n, H), 7.0, device="cuda") if lse is None else lse
    ws = bd.alloc_workspace(bd.latent_attn_workspace_size(d["B"], n, H, R)) if ws is None else ws
    bd.mtp_latent_attn(bd.make_latent_cache(d["pages"], d["table"], d["Dr"]), d["row_start"] if row_start is None else row_start,
                       d["ctx_len"], d["q"], out, lse, ws, d["scale"], window=d["window"], sinks=d["sinks"])
    torch.cuda.synchronize()
    if expect is not None:
        assert bd.get_status(ws) == expect
    return out, lse


def make_prompt(rows, ctx, H, Dn, Dr, Dv, seed, window=0, sinks=0, pad=0, key_pad=0):
    """Queries, and keys and values of every head of contexts and rows; rows of keys that
    belong to no sequence hold NaN."""
    B = len(rows)
    g = torch.Generator(device="cpu").manual_seed(seed)
    total = [c + r for c, r in zip(ctx, rows)]
    start, first = torch.zeros(B + 1, dtype=torch.int32), torch.zeros(B + 1, dtype=torch.int32)
    start[1:] = torch.tensor(rows, dtype=torch.int32).cumsum(0)
    first[1:] = torch.tensor([t + key_pad for t in total], dtype=torch.int32).cumsum(0)
    n_rows, n_keys = max(1, int(start[-1]) + pad), max(1, int(first[-1]))
    kv = torch.randn(n_keys, H, Dn + Dv, generator=g).to(torch.bfloat16)
    k_rope = torch.randn(n_keys, Dr, generator=g).to(torch.bfloat16)
    for b in range(B):
        kv[first[b] + total[b]:first[b + 1]] = float("nan")
        k_rope[first[b] + total[b]:first[b + 1]] = float("nan")
    q = torch.randn(n_rows, H, Dn + Dr, generator=g).to(torch.bfloat16)
    return dict(B=B, H=H, Dn=Dn, Dr=Dr, Dv=Dv, rows=rows, ctx=ctx, window=window, sinks=sinks, n_rows=n_rows, n_keys=n_keys,
                scale=(Dn + Dr) ** -0.5, q=q.cuda(), kv=kv.cuda(), k_rope=k_rope.cuda(), row_start=start.cuda(),
                key_start=first.cuda(), ctx_len=torch.tensor(ctx, dtype=torch.int32).cuda())


def prefill_reference(d):
    n, H, Dn, Dv = d["n_rows"], d["H"], d["Dn"], d["Dv"]
    out, spread = torch.zeros(n, H, Dv, dtype=torch.float64), torch.zeros(n, H, Dv, dtype=torch.float64)
    lse, err = torch.full((n, H), -math.inf, dtype=torch.float64), torch.zeros(n, H, dtype=torch.float64)
    r, first = 0, d["key_start"].tolist()
    for b, m in enumerate(d["rows"]):
        if m:
            at = slice(first[b], first[b] + d["ctx"][b] + m)
            k = torch.cat([d["kv"][at, :, :Dn], d["k_rope"][at, None].expand(-1, H, -1)], dim=-1)
            e = slice(r, r + m)
            out[e], lse[e], spread[e], err[e] = attention(d["q"][e], k, d["kv"][at, :, Dn:],
                                                          sees(d["ctx"][b], m, k.shape[0], d["window"], d["sinks"]), d["scale"])
        r += m
    return out, lse, spread, err


def check_prefill(d, out, lse):
    check_rows(prefill_reference(d), out, lse, sum(d["rows"]), max(c + r for c, r in zip(d["ctx"], d["rows"])))


def prefill(d, out=None, lse=None, ws=None, row_start=None, key_start=None, expect=0):
    """mtp_latent_prefill of the case; (out, lse)."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    n, H, Dv = d["n_rows"], d["H"], d["Dv"]
    out = torch.full((n, H, Dv), 7.0, device="cuda", dtype=torch.bfloat16) if out is None else out
    lse = torch.full((n, H), 7.0, device="cuda") if lse is None else lse
    ws = bd.alloc_workspace(bd.latent_prefill_workspace_size(d["B"], n, H, Dv)) if ws is None else ws
    bd.mtp_latent_prefill(d["row_start"] if row_start is None else row_start, d["ctx_len"],
                          d["key_start"] if key_start is None else key_start, d["q"], d["kv"], d["k_rope"], out, lse, ws,
                          d["scale"], window=d["window"], sinks=d["sinks"])
    torch.cuda.synchronize()
    if expect is not None:
        assert bd.get_status(ws) == expect
    return out, lse


def check_product(x, w, y):
    """y[n, h] = w[h] x[n, h]: K fp32 products and sums, cut off or rounded, then bf16."""
    x, w, got = x.double().cpu().transpose(0, 1), w.double().cpu().transpose(1, 2), y.double().cpu().transpose(0, 1)
    ref, mag = x @ w, x.abs() @ w.abs()
    tol = 2.0 ** -8 * ref.abs() + x.shape[-1] * 2.0 ** -23 * mag * (1 + 2.0 ** -8)
    err = (got - ref).abs()
    assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())


def norm_reference(x, gain, eps):
    x = x.double().cpu()
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * gain.double().cpu()
