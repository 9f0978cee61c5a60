"""The target-side operators around a speculative step, as cases to measure.

Three operators, in the order a serving program runs them for the rows of one
step (k + 1 candidates of every sequence, or a chunk of a prompt):

  append  rotate the new rows' queries and keys to their positions and write
          keys and values into the pages of a paged K/V cache
  attend  attention of those rows over the paged cache: causal, optionally a
          sliding window with a few first positions that stay visible
  logits  penalties for repeated tokens, biases and a grammar mask on the
          target logits of every candidate position

`run` computes the plain form with elementary torch operations, or, where
`own` is true, calls this library.  `exact` computes the same in 64 bits.
"""

import math
import random

import torch

own = False

DEV = "cuda"

# ----------------------------------------------------------------- the cases


def listed():
    att = dict(op="attend", heads=32, kv_heads=8, dim=128, page=64, window=0, sinks=0, pad=0)
    app = dict(op="append", heads=32, kv_heads=8, dim=128, page=64, rot=128, layout="half", stretch=1.0, pad=0)
    log = dict(op="logits", vocab=151936, mask=True, bias=True, prompt=True)
    return [
        # one user: k = 3 drafts and the last token, over the context of a chat
        dict(app, name="append_verify_b1", batch=1, rows_lo=4, rows_hi=4, ctx_lo=4096, ctx_hi=4096),
        # a full serving batch verifying k = 3
        dict(app, name="append_batch_b64", batch=64, rows_lo=4, rows_hi=4, ctx_lo=1024, ctx_hi=8192, pad=8),
        # two chunks of long prompts; part of the head rotates, in interleaved
        # pairs, stretched to a long context; small pages
        dict(app, name="append_chunks_r8190", heads=40, batch=2, rows_lo=4095, rows_hi=4095, ctx_lo=4093,
             ctx_hi=20477, page=16, rot=64, layout="interleaved", stretch=4.0),
        # one user verifying k = 3 over a chat's context: latency
        dict(att, name="attend_verify_b1", batch=1, rows_lo=4, rows_hi=4, ctx_lo=4096, ctx_hi=4096),
        # a full serving batch verifying k = 3, contexts all different
        dict(att, name="attend_batch_b64", batch=64, rows_lo=4, rows_hi=4, ctx_lo=1024, ctx_hi=8192, pad=8),
        # deep chains over long contexts: k = 5, groups of five query heads
        dict(att, name="attend_deep_b32", heads=40, batch=32, rows_lo=6, rows_hi=6, ctx_lo=16384, ctx_hi=16384),
        # very long contexts under a sliding window with four first positions
        # kept; ragged row counts, small heads, small pages
        dict(att, name="attend_window_b16", dim=64, batch=16, rows_lo=1, rows_hi=5, ctx_lo=30011, ctx_hi=65521,
             page=16, window=4096, sinks=4),
        # one chunk of a long prompt: bound by the matrix products
        dict(att, name="attend_chunk_r4096", batch=1, rows_lo=4096, rows_hi=4096, ctx_lo=12288, ctx_hi=12288),
        # chunks of prompts of every length beside sequences that verify a few
        # rows: one call for all
        dict(att, name="attend_mixed_b24", batch=24, rows_lo=1, rows_hi=517, ctx_lo=511, ctx_hi=6007, page=32, pad=3),
        # one user with every rule on: latency
        dict(log, name="logits_b1", batch=1, k=3, hist_lo=4096, hist_hi=4096),
        # a full serving batch: penalties and biases without a grammar
        dict(log, name="logits_batch_b64", batch=64, k=3, hist_lo=1024, hist_hi=8192, mask=False),
        # the largest batch and depth, every rule on
        dict(log, name="logits_b256_k5", batch=256, k=5, hist_lo=64, hist_hi=8192),
    ]


def _log_between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "attend", "attend", "logits"])
    if op == "logits":
        vocab = _log_between(rng, 1000, 256000)
        k = rng.randint(0, 8)
        top = max(1, min(256, (256 * 6 * 151936) // ((k + 1) * vocab)))
        hist = _log_between(rng, 1, 16384)
        return dict(op=op, vocab=vocab, mask=rng.random() < 0.6, bias=rng.random() < 0.6, prompt=rng.random() < 0.7,
                    batch=_log_between(rng, 1, top), k=k, hist_lo=rng.randint(0, hist), hist_hi=hist)
    heads, kv_heads, dim = rng.choice([(32, 8, 128), (40, 8, 128), (16, 2, 64), (2, 2, 32), (24, 8, 128), (14, 2, 64),
                                       (12, 4, 128), (8, 8, 64), (16, 2, 128)])
    case = dict(op=op, heads=heads, kv_heads=kv_heads, dim=dim, page=rng.choice([16, 32, 64, 128]), pad=rng.choice([0, 0, 1, 5]))
    chunk = rng.random() < 0.4
    if chunk:
        batch, rows = _log_between(rng, 1, 6), _log_between(rng, 10, 2048)
        ctx = _log_between(rng, 1, 8192)
        case.update(batch=batch, rows_lo=rng.randint(1, rows), rows_hi=rows, ctx_lo=rng.choice([0, ctx // 2, ctx]), ctx_hi=ctx)
    else:
        batch = _log_between(rng, 1, 64)
        rows = rng.randint(1, 9)
        ctx = _log_between(rng, 1, min(32768, 64 * 8192 // batch))
        case.update(batch=batch, rows_lo=rng.randint(0, rows), rows_hi=rows, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx)
    if op == "append":
        case.update(rot=rng.choice([dim, dim, dim // 2, dim // 4]), layout=rng.choice(["half", "interleaved"]),
                    stretch=rng.choice([1.0, 4.0, 8.0]))
    elif rng.random() < 0.4:
        case.update(window=_log_between(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 70]))
    else:
        case.update(window=0, sinks=0)
    return case


# ----------------------------------------------------------------- the inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _between(lo, hi, n, g):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def _inv_freq(rot, stretch):
    """Radians a position, 64 bits: base^(-2i/rot), and for a stretched context
    the slow half of the pairs divided by the stretch."""
    i = torch.arange(rot // 2, dtype=torch.float64)
    f = 10000.0 ** (-2.0 * i / rot)
    if stretch != 1.0:
        slow = (i / max(1, rot // 2 - 1)).clamp(0, 1)
        f = f * (1.0 - slow) + f / stretch * slow
    return f


def _prepare_cache(case, g):
    B, H, Hkv, D, page = case["batch"], case["heads"], case["kv_heads"], case["dim"], case["page"]
    # how many rows each sequence brings belongs to the case, not to the seed
    pick = random.Random(B)
    rows = torch.tensor([pick.randint(case["rows_lo"], case["rows_hi"]) for _ in range(B)], dtype=torch.int32, device=DEV)
    ctx = _between(case["ctx_lo"], case["ctx_hi"], B, g)
    start = torch.zeros(B + 1, dtype=torch.int32, device=DEV)
    start[1:] = rows.cumsum(0)
    n_rows = max(1, int(start[-1]) + case["pad"])
    need = (ctx.long() + rows.long() + page - 1) // page
    width = (case["ctx_hi"] + case["rows_hi"] + page - 1) // page
    total = B * width
    n_pages = total + 3
    # each sequence's pages in a random order of the pool; -1 past its last
    perm = torch.randperm(n_pages, generator=g, device=DEV)[:total].to(torch.int32)
    first = torch.arange(B, device=DEV) * width
    col = torch.arange(width, device=DEV)
    page_id = perm[first[:, None] + col[None]]
    table = torch.where(col[None] < need[:, None], page_id, torch.full_like(page_id, -1)).contiguous()
    new = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    s = dict(B=B, H=H, Hkv=Hkv, D=D, page=page, n_rows=n_rows, row_start=start, ctx_len=ctx, table=table,
             k_pages=new(n_pages, Hkv, page, D), v_pages=new(n_pages, Hkv, page, D),
             max_rows=max(1, int(rows.max())), l_max=max(1, int((ctx + rows).max())))
    return s, new


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    if op == "logits":
        s = _prepare_logits(case, g)
    else:
        s, new = _prepare_cache(case, g)
        n, H, Hkv, D = s["n_rows"], s["H"], s["Hkv"], s["D"]
        if op == "append":
            # one projection's output holds q, k and v side by side
            s["qkv"] = new(n, (H + 2 * Hkv) * D)
            s["q_out"] = torch.zeros(n, H, D, device=DEV, dtype=torch.bfloat16)
            s["inv_freq"] = _inv_freq(case["rot"], case["stretch"])
            s["cos_scale"] = 1.0 + 0.1 * math.log(case["stretch"])
        else:
            s["q"] = new(n, H, D)
            s["out"] = torch.zeros(n, H, D, device=DEV, dtype=torch.bfloat16)
            s["lse"] = torch.zeros(n, H, device=DEV, dtype=torch.float32)
    s.update(op=op, case=case)
    if own:
        _handles(s)
    return s


def _prepare_logits(case, g):
    B, k, V = case["batch"], case["k"], case["vocab"]
    cap = max(1, case["hist_hi"])
    hist_len = _between(case["hist_lo"], case["hist_hi"], B, g)
    u = torch.rand(B, cap, generator=g, device=DEV)
    # tokens as text has them: a few very often, most seldom
    history = (torch.exp(u * math.log(V)) - 1).to(torch.int32).clamp(0, V - 1)
    u = torch.rand(B, max(1, k), generator=g, device=DEV)
    drafts = (torch.exp(u * math.log(V)) - 1).to(torch.int32).clamp(0, V - 1)
    s = dict(B=B, k=k, V=V, history=history, hist_len=hist_len, drafts=drafts,
             prompt_len=(hist_len // 2).to(torch.int32) if case["prompt"] else torch.zeros_like(hist_len),
             rep=1.0 + 0.3 * torch.rand(B, generator=g, device=DEV), freq=0.5 * torch.rand(B, generator=g, device=DEV),
             pres=0.5 * torch.rand(B, generator=g, device=DEV), bias_tok=None, bias_val=None, bias_len=None, mask=None,
             logits=4.0 * torch.randn(B, k + 1, V, generator=g, device=DEV),
             out=torch.zeros(B, k + 1, V, device=DEV))
    if case["bias"]:
        n = min(64, V)
        s["bias_tok"] = torch.rand(B, V, generator=g, device=DEV).topk(n, dim=1).indices.to(torch.int32).contiguous()
        s["bias_val"] = 5.0 * torch.randn(B, n, generator=g, device=DEV)
        s["bias_len"] = _between(0, n, B, g)
    if case["mask"]:
        words = (V + 31) // 32
        bits = torch.randint(-2**31, 2**31, (B, k + 1, words), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
        more = torch.randint(-2**31, 2**31, (B, k + 1, words), generator=g, device=DEV, dtype=torch.int64).to(torch.int32)
        # free text (everything allowed), a loose grammar, a tight one
        kind = torch.randint(0, 3, (B, k + 1, 1), generator=g, device=DEV)
        bits = torch.where(kind == 0, torch.full_like(bits, -1), torch.where(kind == 1, bits | more, bits & more & (more << 3)))
        s["mask"] = bits.contiguous()
    return s


def _handles(s):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    s["bd"] = bd
    if s["op"] == "logits":
        s["rules"] = bd.make_logit_rules(history=s["history"], prompt_len=s["prompt_len"], hist_len=s["hist_len"], rep=s["rep"],
                                         freq=s["freq"], pres=s["pres"], bias_tok=s["bias_tok"], bias_val=s["bias_val"],
                                         bias_len=s["bias_len"], mask=s["mask"])
        return
    s["cache"] = bd.make_paged_cache(s["k_pages"], s["v_pages"], s["table"])
    if s["op"] == "append":
        layout = bd.ROPE_HALF if s["case"]["layout"] == "half" else bd.ROPE_INTERLEAVED
        s["rope"] = bd.make_rope(bd.rope_table(s["inv_freq"]).to(DEV), s["case"]["rot"], layout, s["cos_scale"])
        s["ws"] = bd.alloc_workspace(256)
    else:
        s["ws"] = bd.alloc_workspace(bd.paged_attn_workspace_size(s["B"], s["n_rows"], s["max_rows"], s["H"], s["Hkv"], s["D"]))


# ----------------------------------------------------------------- one pass


def run(s):
    return {"append": _append, "attend": _attend, "logits": _logits}[s["op"]](s)


def _rows_of(s):
    """Sequence, index within it and position of every real row."""
    at = torch.arange(s["n_rows"], device=DEV)
    b = torch.searchsorted(s["row_start"][1:].long(), at, right=True)
    real = b < s["B"]
    b = b.clamp(max=s["B"] - 1)
    i = at - s["row_start"][b]
    return b, i, s["ctx_len"][b].long() + i, real


def _append(s):
    H, Hkv, D, rot = s["H"], s["Hkv"], s["D"], s["case"]["rot"]
    n = s["n_rows"]
    q, k, v = (x.view(n, -1, D) for x in s["qkv"].split([H * D, Hkv * D, Hkv * D], dim=1))
    if own:
        s["bd"].mtp_cache_append(s["cache"], s["rope"], s["row_start"], s["ctx_len"], q, k, v, s["q_out"], s["ws"])
        return dict(q=s["q_out"], k_pages=s["k_pages"], v_pages=s["v_pages"])
    b, i, pos, real = _rows_of(s)
    # angles of far positions need 64 bits
    angle = pos.double()[:, None] * s["inv_freq"].to(DEV)[None]
    c, sn = (angle.cos() * s["cos_scale"]).float()[:, None], (angle.sin() * s["cos_scale"]).float()[:, None]
    x = torch.cat([q, k], dim=1).float()
    if s["case"]["layout"] == "half":
        x0, x1 = x[..., :rot // 2], x[..., rot // 2:rot]
        y = torch.cat([x0 * c - x1 * sn, x1 * c + x0 * sn, x[..., rot:]], dim=-1)
    else:
        x0, x1 = x[..., 0:rot:2], x[..., 1:rot:2]
        y = torch.cat([torch.stack([x0 * c - x1 * sn, x1 * c + x0 * sn], dim=-1).flatten(-2), x[..., rot:]], dim=-1)
    y = y.to(torch.bfloat16)
    s["q_out"].copy_(torch.where(real[:, None, None], y[:, :H], s["q_out"]))
    page = s["table"][b, (pos // s["page"]).clamp(0, s["table"].shape[1] - 1)].long()[real]
    slot = (pos % s["page"])[real]
    s["k_pages"][page, :, slot] = y[:, H:][real]
    s["v_pages"][page, :, slot] = v[real]
    return dict(q=s["q_out"], k_pages=s["k_pages"], v_pages=s["v_pages"])


def _attend(s):
    B, H, Hkv, D, page = s["B"], s["H"], s["Hkv"], s["D"], s["page"]
    window, sinks = s["case"]["window"], s["case"]["sinks"]
    if own:
        s["bd"].mtp_paged_attn(s["cache"], s["row_start"], s["ctx_len"], s["q"], s["out"], s["lse"], s["ws"], window=window,
                               sinks=sinks, max_rows=s["max_rows"])
        return dict(out=s["out"], lse=s["lse"])
    G, n, L = H // Hkv, s["max_rows"], s["l_max"]
    table = s["table"][:, :(L + page - 1) // page].long().clamp(min=0)
    k = s["k_pages"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)[:, :, :L].float()
    v = s["v_pages"][table].permute(0, 2, 1, 3, 4).reshape(B, Hkv, -1, D)[:, :, :L].float()
    i = torch.arange(n, device=DEV)
    rows = s["row_start"][:-1].long()[:, None] + i[None]
    real = i[None] < (s["row_start"][1:] - s["row_start"][:-1])[:, None]
    q = s["q"][rows.clamp(max=s["n_rows"] - 1)].float()                      # [B, n, H, D]
    q = q.view(B, n, Hkv, G, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, D)
    pos = (s["ctx_len"].long()[:, None] + i[None])[:, :, None]               # [B, n, 1]
    j = torch.arange(L, device=DEV)
    sees = j <= pos
    if window:
        sees = sees & ((j > pos - window) | (j < sinks))
    sc = (q @ k.transpose(-1, -2) / math.sqrt(D)).view(B, Hkv, G, n, L)
    sc = sc.masked_fill(~sees[:, None, None], float("-inf"))
    m = sc.amax(-1, keepdim=True)
    p = (sc - m).exp_()
    l = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, G * n, L) @ v).view(B, Hkv, G, n, D) / l
    o = o.permute(0, 3, 1, 2, 4).reshape(B, n, H, D).to(torch.bfloat16)
    lse = (m + l.log()).squeeze(-1).permute(0, 3, 1, 2).reshape(B, n, H)
    s["out"][rows[real]] = o[real]
    s["lse"][rows[real]] = lse[real]
    return dict(out=s["out"], lse=s["lse"])


def _logits(s):
    if own:
        s["bd"].spec_adjust_logits(s["B"], s["k"], s["V"], s["rules"], s["logits"], s["drafts"], s["out"])
        return s["out"]
    B, k, V = s["B"], s["k"], s["V"]
    at = torch.arange(s["history"].shape[1], device=DEV)[None]
    known = at < s["hist_len"][:, None]
    said = known & (at >= s["prompt_len"][:, None])
    seen = torch.zeros(B, V, device=DEV).scatter_add_(1, s["history"].long(), known.float())
    count = torch.zeros(B, V, device=DEV).scatter_add_(1, s["history"].long(), said.float())
    seen, count = seen[:, None].repeat(1, k + 1, 1), count[:, None].repeat(1, k + 1, 1)
    if k:
        # position j follows the drafts before it
        before = torch.arange(k, device=DEV)[None] < torch.arange(k + 1, device=DEV)[:, None]
        before = before[None].expand(B, -1, -1).float()
        d = s["drafts"].long()[:, None].expand(-1, k + 1, -1)
        seen.scatter_add_(2, d, before)
        count.scatter_add_(2, d, before)
    x = s["logits"]
    r = s["rep"][:, None, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / r, x * r), x)
    x = x - s["freq"][:, None, None] * count - s["pres"][:, None, None] * (count > 0)
    if s["bias_tok"] is not None:
        on = torch.arange(s["bias_tok"].shape[1], device=DEV)[None] < s["bias_len"][:, None]
        bias = torch.zeros(B, V, device=DEV).scatter_add_(1, s["bias_tok"].long(), torch.where(on, s["bias_val"], torch.zeros_like(s["bias_val"])))
        x = x + bias[:, None]
    if s["mask"] is not None:
        t = torch.arange(V, device=DEV)
        allowed = (s["mask"][..., t // 32] >> (t % 32).to(torch.int32)) & 1
        x = x.masked_fill(allowed == 0, float("-inf"))
    s["out"].copy_(x)
    return s["out"]


# ----------------------------------------------------------------- the work


def _sees(first, last, ctx, rows, window, sinks):
    """Keys that some row sees, and (row, key) pairs, of one sequence."""
    if rows == 0:
        return 0, 0
    keys = pairs = 0
    if not window:
        keys, pairs = ctx + rows, rows * ctx + rows * (rows + 1) // 2
        return keys, pairs
    for i in range(rows):
        p = ctx + i
        lo = max(0, p - window + 1)
        pairs += p + 1 - lo + min(sinks, lo)
    lo = max(0, ctx - window + 1)
    return ctx + rows - lo + min(sinks, lo), pairs


def work(case):
    if case["op"] == "logits":
        n = case["batch"] * (case["k"] + 1) * case["vocab"]
        hist = case["batch"] * (case["hist_lo"] + case["hist_hi"]) // 2
        return {"bytes": 8 * n + (n // 8 if case["mask"] else 0) + 4 * hist + (256 * case["batch"] if case["bias"] else 0), "flops": 6 * n}
    B, H, Hkv, D = case["batch"], case["heads"], case["kv_heads"], case["dim"]
    rows, ctx = (case["rows_lo"] + case["rows_hi"]) / 2, (case["ctx_lo"] + case["ctx_hi"]) // 2
    if case["op"] == "append":
        n = B * rows * (H + 2 * Hkv) * D
        return {"bytes": int(4 * n), "flops": int(3 * B * rows * (H + Hkv) * case["rot"])}
    keys, pairs = _sees(0, 0, ctx, int(rows), case["window"], case["sinks"])
    return {"bytes": int(B * (keys * Hkv * D * 4 + rows * H * (4 * D + 4))), "flops": int(B * pairs * 4 * H * D)}


# ----------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _append_exact, "attend": _attend_exact, "logits": _logits_exact}[case["op"]](s)


def _append_exact(s):
    H, Hkv, D, rot = s["H"], s["Hkv"], s["D"], s["case"]["rot"]
    q_out, kp, vp = s["q_out"].double(), s["k_pages"].double(), s["v_pages"].double()
    start, ctx = s["row_start"].tolist(), s["ctx_len"].tolist()
    half = s["case"]["layout"] == "half"
    pairs = torch.arange(rot // 2, device=DEV)
    a, c = (pairs, pairs + rot // 2) if half else (2 * pairs, 2 * pairs + 1)
    for b in range(s["B"]):
        lo, hi = start[b], start[b + 1]
        if hi == lo:
            continue
        pos = torch.arange(ctx[b], ctx[b] + hi - lo, device=DEV)
        turn = torch.polar(torch.full((hi - lo, rot // 2), s["cos_scale"], dtype=torch.float64, device=DEV),
                           torch.outer(pos.double(), s["inv_freq"].to(DEV)))[:, None]
        x = s["qkv"][lo:hi].double().view(hi - lo, H + 2 * Hkv, D)
        qk = x[:, :H + Hkv].clone()
        z = torch.complex(qk[..., a], qk[..., c]) * turn
        qk[..., a], qk[..., c] = z.real, z.imag
        q_out[lo:hi] = qk[:, :H]
        page = s["table"][b].long()[pos // s["page"]]
        kp[page, :, pos % s["page"]] = qk[:, H:]
        vp[page, :, pos % s["page"]] = x[:, H + Hkv:]
    return dict(q=q_out, k_pages=kp, v_pages=vp)


def _attend_exact(s):
    H, Hkv, D, page = s["H"], s["Hkv"], s["D"], s["page"]
    window, sinks = s["case"]["window"], s["case"]["sinks"]
    start, ctx = s["row_start"].tolist(), s["ctx_len"].tolist()
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(s["B"]):
        lo, hi = start[b], start[b + 1]
        if hi == lo:
            continue
        n = hi - lo
        keep = torch.arange(ctx[b] + n, device=DEV)
        if window:
            keep = keep[(keep < sinks) | (keep > ctx[b] - window)]
        where = s["table"][b].long()[keep // page]
        for h in range(Hkv):
            k, v = s["k_pages"][where, h, keep % page].double(), s["v_pages"][where, h, keep % page].double()
            for r in range(0, n, 512):
                m = min(512, n - r)
                mine = slice(h * (H // Hkv), (h + 1) * (H // Hkv))
                q = s["q"][lo + r:lo + r + m, mine].double()
                sc = torch.einsum("ngd,kd->ngk", q, k) * D ** -0.5
                p = torch.arange(ctx[b] + r, ctx[b] + r + m, device=DEV)[:, None]
                hidden = keep[None] > p
                if window:
                    hidden = hidden | ((keep[None] <= p - window) & (keep[None] >= sinks))
                sc = sc.masked_fill(hidden[:, None], -math.inf)
                z = torch.logsumexp(sc, dim=-1)
                out[lo + r:lo + r + m, mine] = torch.einsum("ngk,kd->ngd", (sc - z[..., None]).exp(), v)
                lse[lo + r:lo + r + m, mine] = z
    return dict(out=out, lse=lse)


def _logits_exact(s):
    B, k, V = s["B"], s["k"], s["V"]
    out = torch.empty(B, k + 1, V, dtype=torch.float64, device=DEV)
    hist_len, prompt_len = s["hist_len"].tolist(), s["prompt_len"].tolist()
    bias_len = s["bias_len"].tolist() if s["bias_len"] is not None else None
    shift = torch.arange(32, device=DEV)
    for b in range(B):
        r, f, p = (s[w][b].double() for w in ("rep", "freq", "pres"))
        for j in range(k + 1):
            drafts = s["drafts"][b, :j].long()
            said = torch.cat([s["history"][b, prompt_len[b]:hist_len[b]].long(), drafts]) if prompt_len[b] < hist_len[b] else drafts
            seen = torch.cat([s["history"][b, :hist_len[b]].long(), drafts])
            x = s["logits"][b, j].double()
            ids = seen.unique()
            x[ids] = torch.where(x[ids] > 0, x[ids] / r, x[ids] * r)
            ids, times = said.unique(return_counts=True)
            x[ids] -= f * times + p
            if bias_len is not None:
                x.index_add_(0, s["bias_tok"][b, :bias_len[b]].long(), s["bias_val"][b, :bias_len[b]].double())
            if s["mask"] is not None:
                bits = ((s["mask"][b, j].long()[:, None] >> shift) & 1).flatten()[:V]
                x[bits == 0] = -math.inf
            out[b, j] = x
    return out
