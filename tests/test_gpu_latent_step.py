"""Latent attention as a serving program runs it: a prompt through the expanded form,
then candidate rows through the absorbed one, over the same pages."""

import pytest
import torch

from latent_helpers import attention, attend, check_attend, check_product, check_rows, make_latent, make_prompt, norm_reference, prefill, sees
from paged_helpers import append_reference

pytestmark = pytest.mark.gpu

BF = dict(device="cuda", dtype=torch.bfloat16)


class Layer:
    """One layer's attention, from its projections' outputs to the heads' outputs."""

    def __init__(self, B, H, R, Dr, Dn, Dv, page, ctx_cap, seed):
        from mtp_speculative_decoding_draft_gb300 import binding as bd
        self.bd, self.B, self.H, self.R, self.Dr, self.Dn, self.Dv, self.page = bd, B, H, R, Dr, Dn, Dv, page
        g = self.g = torch.Generator(device="cuda").manual_seed(seed)
        self.up = (torch.randn(H, Dn + Dv, R, generator=g, device="cuda") * R ** -0.5).to(torch.bfloat16)
        self.gain = (1 + 0.2 * torch.randn(R, generator=g, device="cuda")).to(torch.bfloat16)
        width = (ctx_cap + page - 1) // page
        table = torch.randperm(B * width, generator=g, device="cuda").to(torch.int32).view(B, width).contiguous()
        self.pages = torch.full((B * width, page, R + Dr), float("nan"), **BF)
        self.cache = bd.make_latent_cache(self.pages, table, Dr)
        self.freq, _ = bd.rope_frequencies(Dr)
        self.rope = bd.make_rope(bd.rope_table(self.freq).cuda(), Dr, bd.ROPE_INTERLEAVED)
        self.ws = bd.alloc_workspace(256)
        self.scale = (Dn + Dr) ** -0.5

    def rows(self, n):
        g = self.g
        return (torch.randn(n, self.H, self.Dn + self.Dr, generator=g, device="cuda").to(torch.bfloat16),
                torch.randn(n, self.R + self.Dr, generator=g, device="cuda").to(torch.bfloat16))

    def absorbed(self, n):
        """Buffers and the calls of n candidate rows."""
        bd, H, R, Dr, Dn, Dv = self.bd, self.H, self.R, self.Dr, self.Dn, self.Dv
        s = dict(q=torch.zeros(n, H, Dn + Dr, **BF), kv=torch.zeros(n, R + Dr, **BF), ql=torch.zeros(n, H, R + Dr, **BF),
                 ol=torch.zeros(n, H, R, **BF), out=torch.zeros(n, H, Dv, **BF), lse=torch.zeros(n, H, device="cuda"),
                 ws=bd.alloc_workspace(bd.latent_attn_workspace_size(self.B, n, H, R)))

        def run(row_start, ctx_len):
            bd.mtp_latent_append(self.cache, self.rope, row_start, ctx_len, s["kv"], self.gain, 1e-6, s["q"][..., Dn:],
                                 s["ql"][..., R:], self.ws)
            bd.mtp_latent_heads(s["q"][..., :Dn], self.up[:, :Dn].transpose(1, 2), s["ql"][..., :R], self.ws)
            bd.mtp_latent_attn(self.cache, row_start, ctx_len, s["ql"], s["ol"], s["lse"], s["ws"], self.scale)
            bd.mtp_latent_heads(s["ol"], self.up[:, Dn:], s["out"], self.ws)
        return s, run

    def expanded(self, q, kv, row_start, ctx_len, key_start, n_keys):
        """The same rows through every head's own keys and values."""
        bd, H, Dn, Dv, Dr = self.bd, self.H, self.Dn, self.Dv, self.Dr
        n = q.shape[0]
        bd.mtp_latent_append(self.cache, self.rope, row_start, ctx_len, kv, self.gain, 1e-6, q[..., Dn:], q[..., Dn:], self.ws)
        hkv, kr = torch.full((n_keys, H, Dn + Dv), float("nan"), **BF), torch.full((n_keys, Dr), float("nan"), **BF)
        bd.mtp_latent_expand(self.cache, key_start, self.up, hkv, kr, self.ws)
        out, lse = torch.zeros(n, H, Dv, **BF), torch.zeros(n, H, device="cuda")
        ws = bd.alloc_workspace(bd.latent_prefill_workspace_size(self.B, n, H, Dv))
        bd.mtp_latent_prefill(row_start, ctx_len, key_start, q, hkv, kr, out, lse, ws, self.scale)
        torch.cuda.synchronize()
        assert bd.get_status(self.ws) == 0 and bd.get_status(ws) == 0
        return out, lse, hkv, kr

    def latent(self, b, n):
        """The first n cached rows of sequence b, as they are in the pages."""
        j = torch.arange(n)
        table = self.cache.tensors[1].cpu().long()
        return self.pages.cpu()[table[b, j // self.page], j % self.page]


def starts(n):
    s = torch.zeros(len(n) + 1, dtype=torch.int32)
    s[1:] = torch.tensor(n).cumsum(0)
    return s.cuda()


@pytest.mark.parametrize("R,Dr,H,Dn,Dv", [(256, 32, 8, 64, 64), (512, 64, 40, 128, 128)])
@pytest.mark.parametrize("captured", [False, True])
def test_prompt_then_two_verified_steps(R, Dr, H, Dn, Dv, captured):
    B, k, page = 3, 3, 16
    L = Layer(B, H, R, Dr, Dn, Dv, page, 320, seed=R)
    prompt = [150, 1, 40]
    zero = torch.zeros(B, dtype=torch.int32, device="cuda")
    q, kv = L.rows(sum(prompt))
    raw = kv.clone()
    start = starts(prompt)
    out, lse, hkv, kr = L.expanded(q, kv, start, zero, start, sum(prompt))
    r = 0
    for b, n in enumerate(prompt):
        c, e = L.latent(b, n), slice(r, r + n)
        # the cached rows are the normed, rotated ones; the expanded ones their products
        ref = norm_reference(raw[e, :R], L.gain, 1e-6)
        assert ((c[:, :R].double() - ref).abs() <= (2.0 ** -8 + (R / 2 + 8) * 2.0 ** -24) * ref.abs()).all()
        turned, mag = append_reference(raw[e, None, R:], torch.arange(n), L.freq, Dr, False, 1.0)
        assert ((c[:, None, R:].double() - turned).abs() <= 2.0 ** -8 * turned.abs() + 2.0 ** -20 * mag).all()
        check_product(c[:, None, :R].expand(-1, H, -1), L.up, hkv[e])
        assert torch.equal(kr[e].cpu(), c[:, R:])
        r += n

    # ---- candidate rows: k + 1 a sequence, two accepted, then k + 1 more
    n = B * (k + 1)
    s, run = L.absorbed(n)
    rs = torch.arange(0, n + 1, k + 1, device="cuda", dtype=torch.int32)
    ctx = torch.tensor(prompt, dtype=torch.int32, device="cuda")
    if captured:
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            run(rs, ctx)
            stream.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                run(rs, ctx)
    for step in range(2):
        q, kv = L.rows(n)
        s["q"].copy_(q)
        s["kv"].copy_(kv)
        torch.cuda.synchronize()
        graph.replay() if captured else run(rs, ctx)
        torch.cuda.synchronize()
        assert L.bd.get_status(L.ws) == 0 and L.bd.get_status(s["ws"]) == 0
        # each call against its definition on the inputs it had
        check_product(q[..., :Dn], L.up[:, :Dn].transpose(1, 2), s["ql"][..., :R])
        check_product(s["ol"], L.up[:, Dn:], s["out"])
        now = ctx.tolist()
        d = dict(H=H, R=R, Dr=Dr, rows=[k + 1] * B, ctx=now, n_rows=n, q=s["ql"], scale=L.scale, window=0, sinks=0,
                 seqs=[L.latent(b, now[b] + k + 1) for b in range(B)])
        check_attend(d, s["ol"], s["lse"])
        # the expanded form gives the same rows up to what its bf16 steps and these round away
        total = [c + k + 1 for c in now]
        out, lse, hkv, kr = L.expanded(q.clone(), kv, rs, ctx, starts(total), sum(total))
        for b in range(B):
            e, c = slice(b * (k + 1), (b + 1) * (k + 1)), L.latent(b, total[b]).double()
            up = L.up.double().cpu()
            kk = torch.einsum("lr,hdr->lhd", c[:, :R], up)
            qr, _ = append_reference(q[e][..., Dn:], torch.arange(now[b], total[b]), L.freq, Dr, False, 1.0)
            qq = torch.cat([q[e][..., :Dn].double().cpu(), qr], dim=-1)
            key = torch.cat([kk[..., :Dn], c[:, None, R:].expand(-1, H, -1)], dim=-1)
            want, wlse, spread, _ = attention(qq, key, kk[..., Dn:], sees(now[b], k + 1, total[b], 0, 0), L.scale)
            # what bf16 takes from a score: each form rounds products of the query or of the key
            # (2^-8 of every term) and the rotated parts; from a value and from the output alike
            terms = torch.cat([torch.einsum("lr,hdr->lhd", c[:, :R].abs(), up[:, :Dn].abs()), key[..., Dn:].abs()], dim=-1)
            mag = L.scale * torch.einsum("nhd,lhd->nhl", qq.abs(), terms).amax(-1)
            vmag = torch.einsum("lr,hdr->lhd", c[:, :R].abs(), up[:, Dn:].abs()).amax(0)
            tol = (4 * mag * 2.0 ** -8 + 4 * 2.0 ** -8)[..., None] * vmag[None]
            for got in (s["out"][e], out[e]):
                assert ((got.double().cpu() - want).abs() <= tol).all()
            assert ((s["lse"][e].double().cpu() - wlse).abs() <= 4 * mag * 2.0 ** -8 + 1e-4).all()
            assert ((lse[e].double().cpu() - wlse).abs() <= 4 * mag * 2.0 ** -8 + 1e-4).all()
        ctx += 2


def test_streams_side_by_side():
    """Two calls of each kind at once, on streams and workspaces of their own."""
    cases = [make_latent([4, 3], [700, 90], H, 512, 64, 64, seed=H) for H in (16, 128)]
    prompts = [make_prompt([200, 3], [100, 900], 8, 128, 64, 128, seed=i) for i in range(2)]
    alone = [[x.clone() for x in attend(d)] for d in cases] + [[x.clone() for x in prefill(d)] for d in prompts]
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    calls = []
    for d in cases:
        n, H, R = d["n_rows"], d["H"], d["R"]
        out, lse = torch.zeros(n, H, R, **BF), torch.zeros(n, H, device="cuda")
        ws = bd.alloc_workspace(bd.latent_attn_workspace_size(2, n, H, R))
        c = bd.make_latent_cache(d["pages"], d["table"], d["Dr"])
        calls.append((out, lse, lambda d=d, c=c, out=out, lse=lse, ws=ws: bd.mtp_latent_attn(
            c, d["row_start"], d["ctx_len"], d["q"], out, lse, ws, d["scale"])))
    for d in prompts:
        n, H, Dv = d["n_rows"], d["H"], d["Dv"]
        out, lse = torch.zeros(n, H, Dv, **BF), torch.zeros(n, H, device="cuda")
        ws = bd.alloc_workspace(bd.latent_prefill_workspace_size(2, n, H, Dv))
        calls.append((out, lse, lambda d=d, out=out, lse=lse, ws=ws: bd.mtp_latent_prefill(
            d["row_start"], d["ctx_len"], d["key_start"], d["q"], d["kv"], d["k_rope"], out, lse, ws, d["scale"])))
    streams = [torch.cuda.Stream() for _ in calls]
    torch.cuda.synchronize()
    for _ in range(20):
        for st, (_, _, f) in zip(streams, calls):
            with torch.cuda.stream(st):
                f()
    torch.cuda.synchronize()
    for (out, lse, _), (o, z) in zip(calls, alone):
        assert torch.equal(out, o) and torch.equal(lse, z)


def test_a_workspace_serves_call_after_call():
    """Calls of different kinds and sizes one behind the other in one workspace."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    ds = [make_latent([4, 3], [700, 90], 16, 512, 64, 64, seed=1), make_latent([4, 3], [300, 2000], 128, 512, 64, 32, seed=2),
          make_latent([1], [5000], 8, 256, 32, 16, seed=3)]
    alone = [[x.clone() for x in attend(d)] for d in ds]
    ws = bd.alloc_workspace(max(bd.latent_attn_workspace_size(d["B"], d["n_rows"], d["H"], d["R"]) for d in ds))
    for _ in range(3):
        for d, (o, z) in zip(ds, alone):
            out, lse = attend(d, ws=ws)
            assert torch.equal(out, o) and torch.equal(lse, z)


def test_pools_past_32_bits():
    """Pages that begin past 2^32 bytes and 2^31 elements of the pool."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    R, Dr, page, H = 512, 64, 64, 8
    d = make_latent([3, 2], [100, 70], H, R, Dr, page, seed=6)
    far = 2 ** 31 // (page * (R + Dr)) + 5
    small = d["pages"].shape[0]
    pool = torch.zeros(far + small, page, R + Dr, **BF)
    pool[far:] = d["pages"]
    d["pages"], d["table"] = pool, torch.where(d["table"] >= 0, d["table"] + far, d["table"])
    check_attend(d, *attend(d))
    d["H"] = 128
    d["q"] = torch.randn(d["n_rows"], 128, R + Dr, device="cuda").to(torch.bfloat16)
    check_attend(d, *attend(d))
    # expanded, and written
    c = bd.make_latent_cache(pool, d["table"], Dr)
    w, ws = torch.randn(2, 64, R, **BF), bd.alloc_workspace(256)
    kv, kr = torch.zeros(175, 2, 64, **BF), torch.zeros(175, Dr, **BF)
    bd.mtp_latent_expand(c, torch.tensor([0, 103, 175], dtype=torch.int32, device="cuda"), w, kv, kr, ws)
    rows = torch.randn(5, R + Dr, **BF)
    bd.mtp_latent_append(c, None, d["row_start"], d["ctx_len"], rows, None, 0.0, None, None, ws)
    torch.cuda.synchronize()
    assert bd.get_status(ws) == 0
    lat = torch.cat(d["seqs"])
    check_product(lat[:, None, :R].expand(-1, 2, -1), w, kv)
    assert torch.equal(kr.cpu(), lat[:, R:])
    at = [(0, 100), (0, 101), (0, 102), (1, 70), (1, 71)]
    for i, (b, j) in enumerate(at):
        assert torch.equal(pool[int(d["table"][b, j // page]), j % page], rows[i])


def test_keys_and_values_past_32_bits():
    """Expanded keys and values of more than 2^31 elements, and prompts' rows over them."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    R, Dr, H, Dn, Dv, page = 256, 32, 128, 128, 128, 128
    total, ctx, rows = [65700, 300], [65697, 295], [3, 5]
    d = make_latent(rows, ctx, 1, R, Dr, page, seed=8)
    lat = [s.cuda() for s in d["seqs"]]
    n = sum(total)
    w, ws = torch.randn(H, Dn + Dv, R, **BF) / 16, bd.alloc_workspace(256)
    kv, kr = torch.empty(n, H, Dn + Dv, **BF), torch.empty(n, Dr, **BF)
    assert kv.numel() > 2 ** 31
    starts = torch.tensor([0, total[0], n], dtype=torch.int32, device="cuda")
    bd.mtp_latent_expand(bd.make_latent_cache(d["pages"], d["table"], Dr), starts, w, kv, kr, ws)
    torch.cuda.synchronize()
    assert bd.get_status(ws) == 0 and torch.equal(kr, torch.cat(lat)[:, R:])
    check_product(lat[1][:, None, :R].expand(-1, H, -1), w, kv[total[0]:])
    check_product(lat[0][-100:, None, :R].expand(-1, H, -1), w, kv[total[0] - 100:total[0]])
    q = torch.randn(sum(rows), H, Dn + Dr, **BF)
    p = dict(B=2, H=H, Dn=Dn, Dr=Dr, Dv=Dv, n_rows=sum(rows), window=0, sinks=0, scale=(Dn + Dr) ** -0.5, q=q, kv=kv, k_rope=kr,
             row_start=d["row_start"], ctx_len=d["ctx_len"], key_start=starts)
    out, lse = prefill(p)
    r = 0
    for b, m in enumerate(rows):
        at, e, heads = slice(int(starts[b]), int(starts[b + 1])), slice(r, r + m), [0, 63, 127]
        k = torch.cat([kv[at, heads, :Dn], kr[at, None].expand(-1, 3, -1)], dim=-1)
        ref = attention(q[e][:, heads], k, kv[at, heads, Dn:], sees(ctx[b], m, total[b], 0, 0), p["scale"])
        check_rows(ref, out[e][:, heads], lse[e][:, heads], m, total[b])
        r += m
