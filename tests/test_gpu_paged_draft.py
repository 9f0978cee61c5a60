"""mtp_draft_paged / spec_step_paged: the draft chain over a paged cache, with
rotary positions and a window, against the oracle's block in float64."""

import numpy as np
import pytest
import torch

from mtp_speculative_decoding_draft_gb300 import workloads as W
from mtp_speculative_decoding_draft_gb300.model import DraftModule, Verifier, to_device
from oracle.block import linear, rmsnorm, silu
from oracle.numerics import as_f64, bf16_bits_to_f64, round_bf16
from parity_helpers import bf16_ulp_ok, kv_sum_abs, rel_l2

pytestmark = pytest.mark.gpu

GREEDY, STOCH = 0, 1
MID = W.Workload("mid_b3_d256_v5003", B=3, k=4, V=5003, d=256, Hq=4, Hkv=2, Dh=64, F=768, ctx=(1, 200), T=0.8, seed=2001)
GQA5 = W.Workload("gqa5_b2_d640_v3001", B=2, k=2, V=3001, d=640, Hq=10, Hkv=2, Dh=128, F=1280, ctx=(60, 300), T=1.0,
                  seed=2002)
WIDE = W.Workload("wide_b9_d256_v2003", B=9, k=3, V=2003, d=256, Hq=8, Hkv=2, Dh=64, F=512, ctx=(0, 90), T=1.0, seed=2003)


def rotate(x, pos, freq, half):
    """x [..., Dh] float64 at position pos; freq [rot/2] radians a position."""
    n = len(freq)
    a, c = (np.arange(n), np.arange(n) + n) if half else (2 * np.arange(n), 2 * np.arange(n) + 1)
    y = x.copy()
    co, si = np.cos(pos * freq), np.sin(pos * freq)
    y[..., a] = x[..., a] * co - x[..., c] * si
    y[..., c] = x[..., c] * co + x[..., a] * si
    return y


def chain(Wt, w, ctx, forced, rope, window, sinks):
    """Logits [B, k, V], rotated keys and values [B, k, Hkv, Dh] and the attention
    inputs [B, k, d] of the chain fed the GPU's own drafts."""
    B, k, d, Hq, Hkv, Dh = w.B, w.k, w.d, w.Hq, w.Hkv, w.Dh
    logits, ks, vs, ins = np.zeros((B, k, w.V)), np.zeros((B, k, Hkv, Dh)), np.zeros((B, k, Hkv, Dh)), np.zeros((B, k, d))
    rot = lambda x, p: x if rope is None else rotate(x, p, rope[0], rope[1])  # noqa: E731
    for b in range(B):
        L = int(ctx["ctx_len"][b])
        K = bf16_bits_to_f64(ctx["k_cache"][b][:, :L]).copy()
        V = bf16_bits_to_f64(ctx["v_cache"][b][:, :L]).copy()
        x, tok = bf16_bits_to_f64(ctx["h"][b]), int(ctx["last_tok"][b])
        for j in range(k):
            u = np.concatenate([rmsnorm(as_f64(Wt["E"][tok]), Wt["g_emb"], w.eps), rmsnorm(x, Wt["g_hid"], w.eps)])
            x0 = linear(Wt["fc"], u)
            n = rmsnorm(x0, Wt["g_attn"], w.eps)
            q = rot(linear(Wt["wq"], n).reshape(Hq, Dh), L + j)
            kn = round_bf16(rot(round_bf16(linear(Wt["wk"], n)).reshape(Hkv, Dh), L + j))
            vn = round_bf16(linear(Wt["wv"], n)).reshape(Hkv, Dh)
            K, V = np.concatenate([K, kn[:, None]], 1), np.concatenate([V, vn[:, None]], 1)
            t = np.arange(L + j + 1)
            keep = t[(t < sinks) | (t > L + j - window)] if window else t
            o = np.zeros((Hq, Dh))
            for h in range(Hq):
                g = h // (Hq // Hkv)
                s = K[g][keep] @ q[h] / np.sqrt(Dh)
                p = np.exp(s - s.max())
                o[h] = p / p.sum() @ V[g][keep]
            x1 = x0 + linear(Wt["wo"], o.reshape(-1))
            m = rmsnorm(x1, Wt["g_mlp"], w.eps)
            x = x1 + linear(Wt["wdown"], silu(linear(Wt["wgate"], m)) * linear(Wt["wup"], m))
            logits[b, j] = linear(Wt["E"], rmsnorm(x, Wt["g_final"], w.eps))
            ks[b, j], vs[b, j], ins[b, j] = kn, vn, n
            tok = int(forced[b, j])
    return logits, ks, vs, ins


def paged_module(w, ctx, wts, page, rope=None, window=0, sinks=0):
    """A DraftModule whose contexts lie in shuffled pages; slots past the context hold NaN."""
    m = DraftModule(w, wts)
    m.set_context(ctx)
    width = (w.ctx_max + w.k + page - 1) // page
    n = w.B * width + 2
    order = np.random.default_rng(7).permutation(n)[:w.B * width].reshape(w.B, width).astype(np.int32)
    pools = []
    for name in ("k_cache", "v_cache"):
        pool = np.full((n, w.Hkv, page, w.Dh), 0x7fc0, dtype=np.uint16)
        for b in range(w.B):
            for j in range(int(ctx["ctx_len"][b])):
                pool[order[b, j // page], :, j % page] = ctx[name][b][:, j]
        pools.append(torch.from_numpy(pool.view(np.int16)).view(torch.bfloat16).cuda())
    m.set_pages(pools[0], pools[1], to_device(order), rope, window, sinks)
    return m, order


@pytest.mark.parametrize("w", [W.TINY, MID, GQA5, WIDE], ids=lambda w: w.name)
@pytest.mark.parametrize("kind", ["plain", "half", "interleaved", "window"])
def test_chain_matches_the_oracle(w, kind):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    wts, ctx, u = W.make_weights(w), W.make_context(w), W.make_uniforms(w)
    page = 16 if kind == "window" else 64
    rope = freq = None
    if kind != "plain":
        rot = w.Dh if kind != "interleaved" else w.Dh // 2
        freq, _ = bd.rope_frequencies(rot)
        half = kind != "interleaved"
        rope = bd.make_rope(bd.rope_table(freq).cuda(), rot, bd.ROPE_HALF if half else bd.ROPE_INTERLEAVED)
    window, sinks = (9, 2) if kind == "window" else (0, 0)
    m, order = paged_module(w, ctx, wts, page, rope, window, sinks)
    before = [p.clone() for p in (m.cache.tensors[0], m.cache.tensors[1])]
    m.draft_paged(w.T, STOCH, to_device(u["u_draft"]))
    torch.cuda.synchronize()
    assert bd.get_status(m.ws_paged) == 0
    m.check_canaries()
    tok = m.draft_tok.view(w.B, w.k).cpu().numpy()
    got = m.draft_logits.view(w.B, w.k, w.V).cpu().numpy()
    logits, ks, vs, ins = chain(wts, w, ctx, tok, None if rope is None else (freq.numpy(), half), window, sinks)
    for b in range(w.B):
        for j in range(w.k):
            assert rel_l2(got[b, j], logits[b, j]) <= 1e-2, (b, j, rel_l2(got[b, j], logits[b, j]))
    # the appended slots hold the oracle's rows, every other slot is as it was
    for i, (pool, was, ora, name) in enumerate(zip(m.cache.tensors[:2], before, (ks, vs), ("wk", "wv"))):
        now, was = pool.cpu().view(torch.int16).numpy().view(np.uint16), was.cpu().view(torch.int16).numpy().view(np.uint16)
        for b in range(w.B):
            for j in range(w.k):
                pos = int(ctx["ctx_len"][b]) + j
                where = (order[b, pos // page], slice(None), pos % page)
                if j == 0 and (rope is None or name == "wv"):
                    # the first depth's rows see no rounding of this path before them
                    assert bf16_ulp_ok(bf16_bits_to_f64(now[where]), ora[b, j],
                                       kv_sum_abs(wts, ins[b:b + 1, 0])[i][0].reshape(w.Hkv, w.Dh))
                else:
                    assert rel_l2(bf16_bits_to_f64(now[where]), ora[b, j]) <= 1e-2
                was[where] = now[where]
        assert np.array_equal(now, was)


@pytest.mark.parametrize("mode", [GREEDY, STOCH])
def test_step_is_draft_then_verify(mode):
    w = MID
    wts, ctx, u = W.make_weights(w), W.make_context(w), W.make_uniforms(w)
    m, _ = paged_module(w, ctx, wts, 32)
    m.draft_paged(w.T, mode, to_device(u["u_draft"]))
    target = (m.draft_logits.view(w.B, w.k, w.V).new_zeros(w.B, w.k + 1, w.V)
              + to_device(W.target_logits(w)))
    target[:, :w.k] += m.draft_logits.view(w.B, w.k, w.V) * 3
    tok, lg = m.draft_tok.clone(), m.draft_logits.clone()
    v = Verifier(w.B, w.k, w.V)
    ua, uf = to_device(u["u_accept"]), to_device(u["u_final"])
    v(w.T, mode, target, lg, tok, ua, uf)
    m.step_paged(w.T, mode, target, to_device(u["u_draft"]), ua, uf)
    torch.cuda.synchronize()
    assert torch.equal(m.draft_tok, tok) and torch.equal(m.draft_logits, lg)
    out, length, acc = v.results()
    assert np.array_equal(m.out_tok.view(w.B, w.k + 1).cpu().numpy(), out)
    assert np.array_equal(m.accept_len.cpu().numpy(), length) and np.array_equal(m.num_accepted.cpu().numpy(), acc)


def test_a_captured_step_replays():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    w = GQA5
    wts, ctx, u = W.make_weights(w), W.make_context(w), W.make_uniforms(w)
    f, _ = bd.rope_frequencies(w.Dh)
    rope = bd.make_rope(bd.rope_table(f).cuda(), w.Dh)
    m, _ = paged_module(w, ctx, wts, 64, rope)
    target, ud = to_device(W.target_logits(w)), to_device(u["u_draft"])
    ua, uf = to_device(u["u_accept"]), to_device(u["u_final"])
    m.step_paged(w.T, STOCH, target, ud, ua, uf)
    torch.cuda.synchronize()
    want = (m.draft_tok.clone(), m.draft_logits.clone(), m.out_tok.clone())
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        m.step_paged(w.T, STOCH, target, ud, ua, uf)
    for t in (m.draft_tok, m.draft_logits, m.out_tok):
        t.zero_()
    g.replay()
    torch.cuda.synchronize()
    for t, x in zip((m.draft_tok, m.draft_logits, m.out_tok), want):
        assert torch.equal(t, x)


def test_bad_positions_are_flagged():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    w = MID
    m, _ = paged_module(w, W.make_context(w), W.make_weights(w), 64)
    for p in m.cache.tensors[:2]:
        p.nan_to_num_(0.0)
    m.ctx_len.fill_(1 << 20)
    m.draft_paged(w.T, GREEDY)
    assert bd.get_status(m.ws_paged) & bd.STATUS_BAD_CTX
    m.check_canaries()
