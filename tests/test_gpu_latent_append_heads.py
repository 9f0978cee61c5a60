"""mtp_latent_append of queries in either order, rows of heads or heads of rows."""

import pytest
import torch

from latent_helpers import make_latent

pytestmark = pytest.mark.gpu


def part(order, n, H, lead, Dr, fill=None):
    """(whole buffer, its rotary parts [rows, heads, Dr]) with heads within rows or rows within heads."""
    shape = (n, H, lead + Dr) if order == "rows" else (H, n, lead + Dr)
    buf = torch.randn(shape, device="cuda").to(torch.bfloat16) if fill is None else torch.full(shape, fill, device="cuda").bfloat16()
    return buf, buf[..., lead:] if order == "rows" else buf[..., lead:].transpose(0, 1)


@pytest.mark.parametrize("rows,ctx", [([1], [70]), ([3, 0, 5], [0, 9, 300]), ([300, 41], [17, 1000])])
@pytest.mark.parametrize("H,Dr,rot", [(5, 64, 64), (128, 32, 24), (1, 64, 40)])
def test_orders_of_rows_and_heads_give_the_same(rows, ctx, H, Dr, rot):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    torch.manual_seed(len(rows))
    d = make_latent(rows, ctx, 1, 256, Dr, 32, seed=H, pad=2)
    n, m = d["n_rows"], sum(rows)
    kv = torch.randn(n, 256 + Dr, device="cuda").to(torch.bfloat16)
    f, _ = bd.rope_frequencies(rot)
    c = bd.make_latent_cache(d["pages"], d["table"], Dr)
    r = bd.make_rope(bd.rope_table(f).cuda(), rot, bd.ROPE_HALF, 1.0)
    ws = bd.alloc_workspace(256)
    run = lambda q, to: bd.mtp_latent_append(c, r, d["row_start"], d["ctx_len"], kv, None, 0.0, q, to, ws)  # noqa: E731
    x = torch.randn(n, H, Dr, device="cuda").to(torch.bfloat16)
    _, q = part("rows", n, H, 8, Dr)
    q.copy_(x)
    _, want = part("rows", n, H, 0, Dr, 9.0)
    run(q, want)
    pages = d["pages"].clone()
    for frm in ("rows", "heads"):
        for to in ("rows", "heads"):
            _, q = part(frm, n, H, 8, Dr)
            q.copy_(x)
            whole, out = part(to, n, H, 16, Dr, 9.0)
            run(q, out)
            torch.cuda.synchronize()
            assert torch.equal(out, want) and (whole[..., :16] == 9).all() and (out[m:] == 9).all()
        whole, q = part(frm, n, H, 8, Dr)
        q.copy_(x)
        was = whole[..., :8].clone()
        run(q, q)                                              # in place
        torch.cuda.synchronize()
        assert torch.equal(q[:m], want[:m]) and torch.equal(q[m:], x[m:]) and torch.equal(whole[..., :8], was)
    assert bd.get_status(ws) == 0 and torch.equal(d["pages"].view(torch.int16), pages.view(torch.int16))


def test_rows_on_top_of_heads_are_refused():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_latent([4], [0], 1, 256, 64, 32, seed=1)
    c, ws = bd.make_latent_cache(d["pages"], d["table"], 64), bd.alloc_workspace(256)
    kv, buf = (torch.zeros(4096, device="cuda", dtype=torch.bfloat16) for _ in range(2))
    kv = kv[:4 * 320].view(4, 320)
    good = buf[:4 * 2 * 64].view(4, 2, 64)
    for bad in (buf.as_strided((4, 2, 64), (64, 64, 1)), buf.as_strided((4, 2, 64), (64, 248, 1))):
        for q, to in ((bad, good), (good, bad), (bad, bad)):
            with pytest.raises(bd.MtpError):
                bd.mtp_latent_append(c, None, d["row_start"], d["ctx_len"], kv, None, 0.0, q, to, ws)
