"""The target's latent attention around a speculative step, as cases to measure.

A target whose keys and values come from one shared latent vector a token keeps
that vector (R elements) and one rotated key part (Dr elements) for all heads.
Five operators, in the order a serving program runs them:

  append   norm the new rows' latents, rotate their shared key part and the
           queries' rotary parts, write the latent rows into the pages of a cache
  heads    a product a head: queries into the latent space before the absorbed
           attention, its outputs out of it
  attend   absorbed attention of the rows over the paged latents: every head
           reads the same row as key (R + Dr) and as value (its first R)
  expand   keys and values of every head from the cached latents, for a prompt
  prefill  attention of a prompt's rows over those expanded keys and values,
           the rotary key part shared by the heads

`run` computes the plain form with elementary torch operations, or, where
`own` is true, calls this library.  `exact` computes the same in 64 bits.
"""

import math
import random

import torch

own = False

DEV = "cuda"
EPS = 1e-6

# ----------------------------------------------------------------- the cases


def listed():
    geo = dict(rank=512, rope=64, page=64, pad=0)
    app = dict(geo, op="append", heads=128, layout="interleaved", norm=True)
    hd = dict(op="heads", heads=128, nope=128, rank=512)
    att = dict(geo, op="attend", heads=128, window=0, sinks=0)
    exp = dict(geo, op="expand", heads=128, nope=128, value=128)
    pre = dict(op="prefill", heads=32, nope=128, rope=64, value=128, window=0, sinks=0, pad=0)
    return [
        # one user: k = 3 drafts and the last token, over the context of a chat
        dict(app, name="append_verify_b1", batch=1, rows_lo=4, rows_hi=4, ctx_lo=4096, ctx_hi=4096),
        # two chunks of long prompts, halves rotated, small pages
        dict(app, name="append_chunks_r8190", heads=40, layout="half", page=16, batch=2, rows_lo=4095, rows_hi=4095,
             ctx_lo=4093, ctx_hi=20477),
        # one user's attention outputs out of the latent space: latency, bound by the weights
        dict(hd, name="heads_out_b1", way="out", rows=4),
        # queries of a full serving batch that verifies k = 3, into the latent space
        dict(hd, name="heads_in_b64", way="in", rows=256),
        # one user verifying k = 3 over a chat's context: latency
        dict(att, name="attend_verify_b1", batch=1, rows_lo=4, rows_hi=4, ctx_lo=4096, ctx_hi=4096),
        # a full serving batch verifying k = 3, contexts all different: bound by the matrix products
        dict(att, name="attend_batch_b64", batch=64, rows_lo=4, rows_hi=4, ctx_lo=1024, ctx_hi=8192, pad=8),
        # plain decoding of long contexts with few heads: bound by the cache's bytes
        dict(att, name="attend_decode_b32", heads=16, batch=32, rows_lo=1, rows_hi=1, ctx_lo=16384, ctx_hi=32749),
        # chunks of prompts of every length beside sequences that verify a few rows, a smaller
        # latent under a sliding window with four first positions kept
        dict(att, name="attend_mixed_b12", heads=40, rank=256, rope=32, page=32, batch=12, rows_lo=1, rows_hi=517, ctx_lo=511,
             ctx_hi=6007, window=4096, sinks=4, pad=3),
        # a prompt's second chunk: the context's keys and values for every head
        dict(exp, name="expand_k12288", batch=1, keys_lo=12288, keys_hi=12288),
        # several prompts of different lengths, few heads, small pages
        dict(exp, name="expand_ragged_b8", heads=16, page=16, batch=8, keys_lo=33, keys_hi=1021),
        # one chunk of a long prompt: bound by the matrix products
        dict(pre, name="prefill_chunk_r4096", batch=1, rows_lo=4096, rows_hi=4096, ctx_lo=8192, ctx_hi=8192),
        # fresh prompts of every length in one call
        dict(pre, name="prefill_ragged_b16", heads=16, batch=16, rows_lo=1, rows_hi=1021, ctx_lo=0, ctx_hi=0, pad=5),
    ]


def _log_between(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["append", "heads", "attend", "attend", "attend", "expand", "prefill", "prefill"])
    heads = rng.choice([1, 5, 8, 16, 20, 24, 32, 40, 64, 96, 128])
    rank, rope = rng.choice([256, 512, 512]), rng.choice([32, 64, 64])
    nope, value = rng.choice([64, 128, 128]), rng.choice([64, 128, 128])
    if op == "heads":
        rows = _log_between(rng, 1, max(1, 1024 * 128 // heads))
        return dict(op=op, heads=heads, nope=nope, rank=rank, way=rng.choice(["in", "out"]), rows=min(rows, 4096))
    if op == "expand":
        batch = _log_between(rng, 1, 16)
        keys = _log_between(rng, 1, min(12288, 12288 * 128 // heads) // batch)
        return dict(op=op, heads=heads, rank=rank, rope=rope, nope=nope, value=value, page=rng.choice([16, 32, 64, 128]),
                    batch=batch, keys_lo=rng.randint(0, keys), keys_hi=keys, pad=rng.choice([0, 3]))
    case = dict(op=op, heads=heads, rope=rope, pad=rng.choice([0, 0, 1, 5]))
    if op == "prefill":
        case.update(nope=nope, value=value)
    else:
        case.update(rank=rank, page=rng.choice([16, 32, 64, 128]))
    if op == "append":
        batch, rows = _log_between(rng, 1, 64), _log_between(rng, 1, 256)
        ctx = _log_between(rng, 1, 32768)
        case.update(batch=batch, rows_lo=rng.randint(0, rows), rows_hi=rows, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx,
                    layout=rng.choice(["half", "interleaved"]), norm=rng.random() < 0.8)
        return case
    if op == "prefill" or rng.random() < 0.3:
        batch, rows = _log_between(rng, 1, 8), _log_between(rng, 10, 2048)
        ctx = _log_between(rng, 1, 8192)
        case.update(batch=batch, rows_lo=rng.randint(1, rows), rows_hi=rows, ctx_lo=rng.choice([0, ctx // 2, ctx]), ctx_hi=ctx)
    else:
        batch, rows = _log_between(rng, 1, 64), rng.randint(1, 9)
        ctx = _log_between(rng, 1, min(32768, 64 * 8192 // batch))
        case.update(batch=batch, rows_lo=rng.randint(0, rows), rows_hi=rows, ctx_lo=rng.randint(0, ctx), ctx_hi=ctx)
    if rng.random() < 0.3:
        case.update(window=_log_between(rng, 1, 8192), sinks=rng.choice([0, 1, 4, 70]))
    else:
        case.update(window=0, sinks=0)
    # no more work, and no more (row, head, key) scores, than the listed cases have
    while (case["batch"] * case["rows_hi"] * case["heads"] * (case["ctx_hi"] + case["rows_hi"]) > 1.2e9 or
           work(case)["flops"] > 5e11 or work(case)["bytes"] > 8e8):
        if case["batch"] > 1:
            case["batch"] = max(1, case["batch"] // 2)
        elif case["rows_hi"] > 16:
            case.update(rows_lo=case["rows_lo"] // 2, rows_hi=case["rows_hi"] // 2 + 1)
        else:
            case.update(ctx_lo=case["ctx_lo"] // 2, ctx_hi=case["ctx_hi"] // 2 + 1)
    return case


# ----------------------------------------------------------------- the inputs


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _between(lo, hi, n, g):
    return torch.randint(lo, hi + 1, (n,), generator=g, device=DEV, dtype=torch.int32)


def _inv_freq(rot):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return 10000.0 ** (-2.0 * i / rot)


def _starts(n):
    start = torch.zeros(n.numel() + 1, dtype=torch.int32, device=DEV)
    start[1:] = n.cumsum(0)
    return start


def _counts(lo, hi, n):
    """How many rows each sequence brings belongs to the case, not to the seed."""
    pick = random.Random(n)
    return torch.tensor([pick.randint(lo, hi) for _ in range(n)], dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    op, H = case["op"], case["heads"]
    new = lambda *shape: torch.randn(shape, generator=g, device=DEV, dtype=torch.bfloat16)  # noqa: E731
    s = dict(op=op, case=case, H=H)
    if op == "heads":
        n, nope, rank = case["rows"], case["nope"], case["rank"]
        # the up projection as a checkpoint holds it: of each head nope rows for keys, then rows for values
        s["up"] = (new(H, 2 * nope, rank).float() * rank ** -0.5).to(torch.bfloat16)
        if case["way"] == "in":
            # queries keep a rotary part behind the part that goes into the latent space
            s["x"] = new(n, H, nope + 64)[..., :nope]
            s["w"] = s["up"][:, :nope].transpose(1, 2)
            s["y"] = torch.zeros(n, H, rank + 64, device=DEV, dtype=torch.bfloat16)[..., :rank]
        else:
            s["x"] = new(n, H, rank)
            s["w"] = s["up"][:, nope:]
            s["y"] = torch.zeros(n, H, nope, device=DEV, dtype=torch.bfloat16)
        if own:
            _handles(s)
        return s
    B = s["B"] = case["batch"]
    if op == "expand":
        n = _counts(case["keys_lo"], case["keys_hi"], B)
        ctx, s["key_start"] = torch.zeros_like(n), _starts(n)
        s["n_keys"] = max(1, int(s["key_start"][-1]) + case["pad"])
        width_of = case["keys_hi"]
    else:
        n = _counts(case["rows_lo"], case["rows_hi"], B)
        ctx = _between(case["ctx_lo"], case["ctx_hi"], B, g)
        s.update(row_start=_starts(n), ctx_len=ctx)
        s["n_rows"] = max(1, int(s["row_start"][-1]) + case["pad"])
        s["max_rows"] = max(1, int(n.max()))
        s["l_max"] = max(1, int((ctx + n).max()))
        width_of = case["ctx_hi"] + case["rows_hi"]
    Dr = case["rope"]
    if op == "prefill":
        nope, value = case["nope"], case["value"]
        s["key_start"] = _starts(ctx + n)
        s["n_keys"] = max(1, int(s["key_start"][-1]))
        s.update(q=new(s["n_rows"], H, nope + Dr), kv=new(s["n_keys"], H, nope + value), k_rope=new(s["n_keys"], Dr),
                 out=torch.zeros(s["n_rows"], H, value, device=DEV, dtype=torch.bfloat16),
                 lse=torch.zeros(s["n_rows"], H, device=DEV), scale=(nope + Dr) ** -0.5)
        if own:
            _handles(s)
        return s
    page, R = case["page"], case["rank"]
    s.update(page=page, R=R)
    need = (ctx.long() + n.long() + page - 1) // page
    width = max(1, (width_of + page - 1) // page)
    total = B * width
    n_pages = total + 3
    # each sequence's pages in a random order of the pool; -1 past its last
    perm = torch.randperm(n_pages, generator=g, device=DEV)[:total].to(torch.int32)
    col = torch.arange(width, device=DEV)
    page_id = perm[(torch.arange(B, device=DEV) * width)[:, None] + col[None]]
    s["table"] = torch.where(col[None] < need[:, None], page_id, torch.full_like(page_id, -1)).contiguous()
    s["pages"] = new(n_pages, page, R + Dr)
    if op == "append":
        s["kv"] = new(s["n_rows"], R + Dr) * 3
        s["gain"] = (1 + 0.2 * torch.randn(R, generator=g, device=DEV)).to(torch.bfloat16) if case["norm"] else None
        s["q"] = new(s["n_rows"], H, 128 + Dr)[..., 128:]
        s["q_out"] = torch.zeros(s["n_rows"], H, R + Dr, device=DEV, dtype=torch.bfloat16)[..., R:]
        s["inv_freq"] = _inv_freq(Dr)
    elif op == "attend":
        s.update(q=new(s["n_rows"], H, R + Dr), out=torch.zeros(s["n_rows"], H, R, device=DEV, dtype=torch.bfloat16),
                 lse=torch.zeros(s["n_rows"], H, device=DEV), scale=(R + Dr) ** -0.5)
    else:
        N = case["nope"] + case["value"]
        s["w"] = (new(H, N, R).float() * R ** -0.5).to(torch.bfloat16)
        s["kv"] = torch.zeros(s["n_keys"], H, N, device=DEV, dtype=torch.bfloat16)
        s["k_rope"] = torch.zeros(s["n_keys"], Dr, device=DEV, dtype=torch.bfloat16)
    if own:
        _handles(s)
    return s


def _handles(s):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    s["bd"] = bd
    op, case = s["op"], s["case"]
    size = 256
    if op in ("append", "attend", "expand"):
        s["cache"] = bd.make_latent_cache(s["pages"], s["table"], case["rope"])
    if op == "append":
        layout = bd.ROPE_HALF if case["layout"] == "half" else bd.ROPE_INTERLEAVED
        s["rope"] = bd.make_rope(bd.rope_table(s["inv_freq"]).to(DEV), case["rope"], layout, 1.0)
    elif op == "attend":
        size = bd.latent_attn_workspace_size(s["B"], s["n_rows"], s["H"], s["R"])
    elif op == "prefill":
        size = bd.latent_prefill_workspace_size(s["B"], s["n_rows"], s["H"], case["value"])
    s["ws"] = bd.alloc_workspace(size)


# ----------------------------------------------------------------- one pass


def run(s):
    return {"append": _append, "heads": _heads, "attend": _attend, "expand": _expand, "prefill": _prefill}[s["op"]](s)


def _rows_of(start, count, B):
    """Sequence, index within it and whether it is one, of `count` rows."""
    at = torch.arange(count, device=DEV)
    b = torch.searchsorted(start[1:].long(), at, right=True)
    real = b < B
    b = b.clamp(max=B - 1)
    return b, at - start[b], real


def _append(s):
    R = s["R"]
    if own:
        s["bd"].mtp_latent_append(s["cache"], s["rope"], s["row_start"], s["ctx_len"], s["kv"], s["gain"], EPS, s["q"], s["q_out"],
                                  s["ws"])
        return dict(q=s["q_out"], pages=s["pages"])
    b, i, real = _rows_of(s["row_start"], s["n_rows"], s["B"])
    pos = s["ctx_len"][b].long() + i
    # angles of far positions need 64 bits
    angle = pos.double()[:, None] * s["inv_freq"].to(DEV)[None]
    c, sn = angle.cos().float()[:, None], angle.sin().float()[:, None]
    x = torch.cat([s["q"], s["kv"][:, None, R:]], dim=1).float()
    if s["case"]["layout"] == "half":
        x0, x1 = x.chunk(2, dim=-1)
        y = torch.cat([x0 * c - x1 * sn, x1 * c + x0 * sn], dim=-1)
    else:
        x0, x1 = x[..., 0::2], x[..., 1::2]
        y = torch.stack([x0 * c - x1 * sn, x1 * c + x0 * sn], dim=-1).flatten(-2)
    y = y.to(torch.bfloat16)
    latent = s["kv"][:, :R].float()
    if s["gain"] is not None:
        latent = latent * torch.rsqrt(latent.square().mean(-1, keepdim=True) + EPS) * s["gain"].float()
    s["q_out"].copy_(torch.where(real[:, None, None], y[:, :-1], s["q_out"]))
    page = s["table"][b, (pos // s["page"]).clamp(0, s["table"].shape[1] - 1)].long()[real]
    s["pages"][page, (pos % s["page"])[real]] = torch.cat([latent.to(torch.bfloat16), y[:, -1]], dim=-1)[real]
    return dict(q=s["q_out"], pages=s["pages"])


def _heads(s):
    if own:
        s["bd"].mtp_latent_heads(s["x"], s["w"], s["y"], s["ws"])
        return s["y"]
    y = s["x"].float().transpose(0, 1) @ s["w"].float().transpose(1, 2)
    s["y"].copy_(y.transpose(0, 1))
    return s["y"]


def _sees(pos, j, window, sinks):
    sees = j <= pos
    if window:
        sees = sees & ((j > pos - window) | (j < sinks))
    return sees


def _block(s, width):
    """The rows of every sequence side by side, [B, n] of them."""
    i = torch.arange(s["max_rows"], device=DEV)
    rows = s["row_start"][:-1].long()[:, None] + i[None]
    real = i[None] < (s["row_start"][1:] - s["row_start"][:-1])[:, None]
    q = s["q"][rows.clamp(max=s["n_rows"] - 1)].float()
    pos = s["ctx_len"].long()[:, None] + i[None]
    sees = _sees(pos[:, :, None], torch.arange(s["l_max"], device=DEV), s["case"]["window"], s["case"]["sinks"])
    return rows, real, q, sees


def _softmax(sc, sees):
    """Weights and log-sums; a row that sees nothing: zeros and -inf."""
    sc = sc.masked_fill(~sees, float("-inf"))
    m = sc.amax(-1, keepdim=True)
    p = (sc - m.clamp(min=-3e38)).exp_()
    l = p.sum(-1, keepdim=True)
    return p, l.clamp(min=1e-37), (m + l.log()).squeeze(-1)


def _attend(s):
    B, H, R, page = s["B"], s["H"], s["R"], s["page"]
    if own:
        s["bd"].mtp_latent_attn(s["cache"], s["row_start"], s["ctx_len"], s["q"], s["out"], s["lse"], s["ws"], s["scale"],
                                window=s["case"]["window"], sinks=s["case"]["sinks"])
        return dict(out=s["out"], lse=s["lse"])
    n, L = s["max_rows"], s["l_max"]
    rows, real, q, sees = _block(s, R)
    table = s["table"][:, :(L + page - 1) // page].long().clamp(min=0)
    k = s["pages"][table].reshape(B, -1, s["pages"].shape[-1])[:, :L].float()
    sc = (q.reshape(B, n * H, -1) @ k.transpose(1, 2) * s["scale"]).view(B, n, H, L)
    p, l, lse = _softmax(sc, sees[:, :, None])
    o = (p.view(B, n * H, L) @ k[..., :R]).view(B, n, H, R) / l
    s["out"][rows[real]] = o[real].to(torch.bfloat16)
    s["lse"][rows[real]] = lse[real]
    return dict(out=s["out"], lse=s["lse"])


def _expand(s):
    if own:
        s["bd"].mtp_latent_expand(s["cache"], s["key_start"], s["w"], s["kv"], s["k_rope"], s["ws"])
        return dict(kv=s["kv"], k_rope=s["k_rope"])
    H, R, page = s["H"], s["R"], s["page"]
    b, j, real = _rows_of(s["key_start"], s["n_keys"], s["B"])
    row = s["pages"][s["table"][b, (j // page).clamp(max=s["table"].shape[1] - 1)].long().clamp(min=0), j % page]
    kv = row[:, :R].float() @ s["w"].float().view(-1, R).t()
    s["kv"].copy_(torch.where(real[:, None, None], kv.view(s["n_keys"], H, -1).to(torch.bfloat16), s["kv"]))
    s["k_rope"].copy_(torch.where(real[:, None], row[:, R:], s["k_rope"]))
    return dict(kv=s["kv"], k_rope=s["k_rope"])


def _prefill(s):
    B, H, nope = s["B"], s["H"], s["case"]["nope"]
    if own:
        s["bd"].mtp_latent_prefill(s["row_start"], s["ctx_len"], s["key_start"], s["q"], s["kv"], s["k_rope"], s["out"], s["lse"],
                                   s["ws"], s["scale"], window=s["case"]["window"], sinks=s["case"]["sinks"])
        return dict(out=s["out"], lse=s["lse"])
    L = s["l_max"]
    rows, real, q, sees = _block(s, nope)
    at = (s["key_start"][:-1].long()[:, None] + torch.arange(L, device=DEV)[None]).clamp(max=s["n_keys"] - 1)
    kv = s["kv"][at].float().transpose(1, 2)                        # [B, H, L, nope + value]
    q = q.transpose(1, 2)                                           # [B, H, n, nope + rope]
    sc = q[..., :nope] @ kv[..., :nope].transpose(-1, -2)
    sc += q[..., nope:] @ s["k_rope"][at].float()[:, None].transpose(-1, -2)
    p, l, lse = _softmax(sc.mul_(s["scale"]), sees[:, None])
    o = ((p @ kv[..., nope:]) / l).transpose(1, 2)
    s["out"][rows[real]] = o[real].to(torch.bfloat16)
    s["lse"][rows[real]] = lse.transpose(1, 2)[real]
    return dict(out=s["out"], lse=s["lse"])


# ----------------------------------------------------------------- the work


def _seen(ctx, rows, window, sinks):
    """Keys that some row sees, and (row, key) pairs, of one sequence."""
    if rows == 0:
        return 0, 0
    if not window:
        return ctx + rows, rows * ctx + rows * (rows + 1) // 2
    pairs = 0
    for i in range(rows):
        p = ctx + i
        lo = max(0, p - window + 1)
        pairs += p + 1 - lo + min(sinks, lo)
    lo = max(0, ctx - window + 1)
    return ctx + rows - lo + min(sinks, lo), pairs


def _mean_counts(lo, hi, n):
    pick = random.Random(n)
    return [pick.randint(lo, hi) for _ in range(n)]


def work(case):
    op, H = case["op"], case["heads"]
    if op == "heads":
        n, K, N = case["rows"], case["nope"], case["rank"]
        return {"bytes": 2 * H * (K * N + n * (K + N)), "flops": 2 * n * H * K * N}
    if op == "expand":
        n, N, R = sum(_mean_counts(case["keys_lo"], case["keys_hi"], case["batch"])), case["nope"] + case["value"], case["rank"]
        return {"bytes": 2 * (n * (R + 2 * case["rope"]) + H * N * (R + n)), "flops": 2 * n * H * N * R}
    counts = _mean_counts(case["rows_lo"], case["rows_hi"], case["batch"])
    n, ctx, Dr = sum(counts), (case["ctx_lo"] + case["ctx_hi"]) // 2, case["rope"]
    if op == "append":
        return {"bytes": 4 * n * (H * Dr + case["rank"] + Dr), "flops": 3 * n * (H + 1) * Dr + 4 * n * case["rank"]}
    seen = [_seen(ctx, r, case["window"], case["sinks"]) for r in counts]
    keys, pairs = sum(k for k, _ in seen), sum(p for _, p in seen)
    if op == "attend":
        R = case["rank"]
        return {"bytes": 2 * keys * (R + Dr) + n * H * (2 * (2 * R + Dr) + 4), "flops": 2 * pairs * H * (2 * R + Dr)}
    D, Dv = case["nope"] + Dr, case["value"]
    return {"bytes": 2 * keys * (H * (case["nope"] + Dv) + Dr) + n * H * (2 * (D + Dv) + 4), "flops": 2 * pairs * H * (D + Dv)}


# ----------------------------------------------------------------- the definition in 64 bits


def exact(case, seed):
    s = prepare(case, seed)
    return {"append": _append_exact, "heads": _heads_exact, "attend": _attend_exact, "expand": _expand_exact,
            "prefill": _prefill_exact}[case["op"]](s)


def _append_exact(s):
    R, Dr = s["R"], s["case"]["rope"]
    q_out, pages = s["q_out"].double(), s["pages"].double()
    start, ctx = s["row_start"].tolist(), s["ctx_len"].tolist()
    pairs = torch.arange(Dr // 2, device=DEV)
    a, c = (pairs, pairs + Dr // 2) if s["case"]["layout"] == "half" else (2 * pairs, 2 * pairs + 1)
    for b in range(s["B"]):
        lo, hi = start[b], start[b + 1]
        if hi == lo:
            continue
        pos = torch.arange(ctx[b], ctx[b] + hi - lo, device=DEV)
        turn = torch.polar(torch.ones(hi - lo, Dr // 2, dtype=torch.float64, device=DEV),
                           torch.outer(pos.double(), s["inv_freq"].to(DEV)))[:, None]
        for x, to in ((s["q"][lo:hi].double(), None), (s["kv"][lo:hi, None, R:].double(), pos)):
            y = x.clone()
            z = torch.complex(x[..., a], x[..., c]) * turn
            y[..., a], y[..., c] = z.real, z.imag
            if to is None:
                q_out[lo:hi] = y
            else:
                key = y[:, 0]
        latent = s["kv"][lo:hi, :R].double()
        if s["gain"] is not None:
            latent = latent / ((latent * latent).sum(-1, keepdim=True) / R + EPS).sqrt() * s["gain"].double()
        pages[s["table"][b].long()[pos // s["page"]], pos % s["page"]] = torch.cat([latent, key], dim=-1)
    return dict(q=q_out, pages=pages)


def _heads_exact(s):
    return torch.stack([s["x"][:, h].double() @ s["w"][h].double().t() for h in range(s["H"])], dim=1)


def _one(q, k, v, pos, s):
    """Attention of rows q [n, D] at positions pos over keys 0 .. of one head."""
    j = torch.arange(k.shape[0], device=DEV)
    hidden = j[None] > pos[:, None]
    if s["case"]["window"]:
        hidden = hidden | ((j[None] <= pos[:, None] - s["case"]["window"]) & (j[None] >= s["case"]["sinks"]))
    sc = (q @ k.t() * s["scale"]).masked_fill(hidden, -math.inf)
    z = torch.logsumexp(sc, dim=-1)
    w = torch.where(torch.isinf(z)[:, None], torch.zeros_like(sc), (sc - z[:, None]).exp())
    return w @ v, z


def _attend_exact(s):
    R, H, page = s["R"], s["H"], s["page"]
    start, ctx = s["row_start"].tolist(), s["ctx_len"].tolist()
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(s["B"]):
        lo, hi = start[b], start[b + 1]
        if hi == lo:
            continue
        j = torch.arange(ctx[b] + hi - lo, device=DEV)
        k = s["pages"][s["table"][b].long()[j // page], j % page].double()
        for r in range(lo, hi, 64):
            e = min(hi, r + 64)
            pos = (torch.arange(r, e, device=DEV) - lo + ctx[b]).repeat_interleave(H)
            o, z = _one(s["q"][r:e].double().reshape(-1, k.shape[1]), k, k[:, :R], pos, s)
            out[r:e], lse[r:e] = o.view(e - r, H, R), z.view(e - r, H)
    return dict(out=out, lse=lse)


def _expand_exact(s):
    R, H, page = s["R"], s["H"], s["page"]
    kv, k_rope = s["kv"].double(), s["k_rope"].double()
    start = s["key_start"].tolist()
    w = s["w"].double().view(-1, R)
    for b in range(s["B"]):
        for r in range(start[b], start[b + 1], 2048):
            e = min(start[b + 1], r + 2048)
            j = torch.arange(r, e, device=DEV) - start[b]
            row = s["pages"][s["table"][b].long()[j // page], j % page].double()
            kv[r:e] = torch.einsum("kr,nr->kn", row[:, :R], w).view(e - r, H, -1)
            k_rope[r:e] = row[:, R:]
    return dict(kv=kv, k_rope=k_rope)


def _prefill_exact(s):
    H, nope = s["H"], s["case"]["nope"]
    start, first, ctx = s["row_start"].tolist(), s["key_start"].tolist(), s["ctx_len"].tolist()
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(s["B"]):
        lo, hi = start[b], start[b + 1]
        keys = slice(first[b], first[b] + ctx[b] + hi - lo)
        for h in range(H if hi > lo else 0):
            k = torch.cat([s["kv"][keys, h, :nope], s["k_rope"][keys]], dim=-1).double()
            v = s["kv"][keys, h, nope:].double()
            for r in range(lo, hi, 2048):
                e = min(hi, r + 2048)
                out[r:e, h], lse[r:e, h] = _one(s["q"][r:e, h].double(), k, v, torch.arange(r, e, device=DEV) - lo + ctx[b], s)
    return dict(out=out, lse=lse)
