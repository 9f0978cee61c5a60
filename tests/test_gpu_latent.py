"""The latent-attention operators against their definitions in 64 bits."""

import pytest
import torch

from latent_helpers import (attend, attention, check_attend, check_prefill, check_product, check_rows, make_latent, make_prompt,
                            norm_reference, prefill, sees)
from paged_helpers import append_reference

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------- append


def run_append(d, rot, half=True, scale=1.0, eps=1e-6, gain=True, in_place=False, with_q=True, rope=True, seed=1, expect=0,
               check=True):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    n, H, R, Dr = d["n_rows"], d["H"], d["R"], d["Dr"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    wide = rnd(n, R + Dr + 40)                             # one projection's output among others
    kv = wide[:, 8:8 + R + Dr]
    whole = rnd(n, H, 96 + Dr)
    q = whole[..., 96:]
    was_q, was = whole.clone(), d["pages"].clone()
    to = whole if in_place else torch.full((n, H, R + Dr), 9.0, device="cuda", dtype=torch.bfloat16)
    was_to = to.clone()
    q_out = q if in_place else to[..., R:]
    gn = (1 + 0.3 * torch.randn(R, generator=g, device="cuda")).to(torch.bfloat16) if gain else None
    f, _ = bd.rope_frequencies(rot)
    r = bd.make_rope(bd.rope_table(f).cuda(), rot, bd.ROPE_HALF if half else bd.ROPE_INTERLEAVED, scale) if rope else None
    ws = bd.alloc_workspace(256)
    bd.mtp_latent_append(bd.make_latent_cache(d["pages"], d["table"], Dr), r, d["row_start"], d["ctx_len"], kv, gn, eps,
                         q if with_q else None, q_out if with_q else None, ws)
    torch.cuda.synchronize()
    assert bd.get_status(ws) == expect
    if not check:
        return was
    m = sum(d["rows"])
    pos = torch.cat([torch.arange(c, c + r) for c, r in zip(d["ctx"], d["rows"])])
    seq = torch.cat([torch.full((r,), b) for b, r in enumerate(d["rows"])]).long()
    if not rope:
        f, scale = torch.zeros_like(f), 1.0

    def turned(got, x):
        ref, mag = append_reference(x, pos, f, rot, half, scale)
        if not rope:
            ref = x.double().cpu()
        # rounded to bf16 (2^-8); sine and cosine of an angle off by 2^-25 of a half turn,
        # good to 2 ulp, the two products and their sum: 2^-20 in all
        err, tol = (got.double().cpu() - ref).abs(), 2.0 ** -8 * ref.abs() + 2.0 ** -20 * mag
        assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())

    if with_q:
        turned(q_out[:m], was_q[:m, :, 96:])
    now = to.clone()                                       # nothing else of the queries changes
    if with_q:
        now[:m, :, -Dr:] = was_to[:m, :, -Dr:]
    assert torch.equal(now, was_to)
    page, slot = d["table"].cpu()[seq, pos // d["page"]].long(), pos % d["page"]
    row = d["pages"].cpu()[page, slot]
    turned(row[:, None, R:], kv[:m, None, R:])
    if gain:
        ref = norm_reference(kv[:m, :R], gn, eps)
        # the sum of squares (R terms, half of its error in the root), the root, the quotient, two products; bf16
        tol = (2.0 ** -8 + (R / 2 + 8) * 2.0 ** -24) * ref.abs()
        assert ((row[:, :R].double() - ref).abs() <= tol).all()
    else:
        assert torch.equal(row[:, :R], kv[:m, :R].cpu())
    a, b = d["pages"].cpu().clone(), was.cpu().clone()     # every other slot is as it was
    a[page, slot] = 0
    b[page, slot] = 0
    assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    return was


@pytest.mark.parametrize("H,R,Dr", [(1, 256, 32), (5, 512, 64), (40, 256, 64), (128, 512, 64), (128, 512, 32)])
@pytest.mark.parametrize("half", [True, False])
def test_append_layouts(H, R, Dr, half):
    run_append(make_latent([1, 0, 5, 3], [0, 7, 62, 300], H, R, Dr, 64, seed=H, pad=2), Dr, half, 1.2)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_append_pages(page):
    run_append(make_latent([40, 1, 17], [page - 1, page, 3 * page + 5], 8, 256, 64, page, seed=page), 64)


@pytest.mark.parametrize("rot", [8, 16, 24, 40, 48, 56])
@pytest.mark.parametrize("half", [True, False])
def test_append_rotates_a_part(rot, half):
    run_append(make_latent([3, 2], [11, 90], 6, 256, 64, 32, seed=rot), rot, half)


def test_append_variants():
    case = lambda s=1: make_latent([2, 6], [5, 100], 8, 512, 64, 64, seed=s, pad=1)  # noqa: E731
    run_append(case(), 64, in_place=True)
    run_append(case(), 64, half=False, in_place=True)
    run_append(case(), 64, with_q=False)
    run_append(case(), 64, rope=False)
    run_append(case(), 64, gain=False)
    run_append(case(), 64, gain=False, rope=False, with_q=False)
    run_append(case(), 64, eps=0.5)


def test_append_many_rows_and_sequences():
    rows = [(i * 5) % 7 for i in range(900)]
    run_append(make_latent(rows, [(i * 13) % 50 for i in range(900)], 2, 256, 32, 16, seed=2, pad=4), 32)


def test_append_flags_and_drops_what_has_no_place():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_latent([4], [62], 4, 256, 64, 64, seed=3)
    d["table"][0, 1] = 1000
    was = run_append(d, 64, expect=bd.STATUS_BAD_PAGE, check=False)
    same = (d["pages"].view(torch.int16) == was.view(torch.int16)).all(-1)
    page = int(d["table"][0, 0])
    assert same.sum() == same.numel() - 2 and not same[page, 62] and not same[page, 63]
    for bad in (1 << 25, -1, 2 ** 31 - 1, -2 ** 31):
        d["ctx_len"].fill_(bad)
        was = run_append(d, 64, expect=bd.STATUS_BAD_CTX, check=False)
        assert torch.equal(d["pages"].view(torch.int16), was.view(torch.int16))
    d["ctx_len"].fill_(0)
    d["row_start"].copy_(torch.tensor([2, 400], dtype=torch.int32))
    run_append(d, 64, expect=bd.STATUS_BAD_ROWS, check=False)


# ------------------------------------------------------------- products


def product(n, H, K, N, transposed, seed=0, order="rows", expect=0):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    from mtp_speculative_decoding_draft_gb300.model import Guarded
    g = torch.Generator(device="cuda").manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    x = rnd(n, H, K + 24)[..., 16:16 + K] if order == "rows" else rnd(H, n, K).transpose(0, 1)
    w = rnd(H, K, N + 8)[..., :N].transpose(1, 2) if transposed else rnd(H, N + 3, K + 8)[:, 3:, :K]
    guard = Guarded()
    if order == "rows":
        buf = guard.alloc("y", n * H * (N + 16), torch.bfloat16).view(n, H, N + 16)
        y = buf[..., 8:8 + N]
    else:
        buf = guard.alloc("y", n * H * N, torch.bfloat16).view(H, n, N)
        y = buf.transpose(0, 1)
    buf.fill_(5.0)
    ws = bd.alloc_workspace(256)
    bd.mtp_latent_heads(x, w, y, ws)
    torch.cuda.synchronize()
    guard.check()
    assert bd.get_status(ws) == expect
    check_product(x, w, y)
    if order == "rows":
        assert (buf[..., :8] == 5).all() and (buf[..., 8 + N:] == 5).all()


@pytest.mark.parametrize("n", [1, 4, 127, 128, 129, 300])
@pytest.mark.parametrize("K,N,transposed", [(128, 512, True), (512, 128, False), (64, 256, True), (256, 64, False)])
def test_products(n, K, N, transposed):
    product(n, 3, K, N, transposed, seed=n)


@pytest.mark.parametrize("K,N", [(8, 8), (40, 24), (72, 136), (200, 1000), (1032, 264)])
@pytest.mark.parametrize("transposed", [True, False])
@pytest.mark.parametrize("order", ["rows", "heads"])
def test_products_of_odd_sizes(K, N, transposed, order):
    product(37, 5, K, N, transposed, seed=K, order=order)


def test_products_of_many_heads():
    product(4, 128, 128, 512, True)
    product(70, 128, 512, 128, False)
    product(2, 1000, 16, 16, False)


def expanded(d, keys, H, N, pad=0, seed=0, key_start=None, expect=0):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    from mtp_speculative_decoding_draft_gb300.model import Guarded
    R, Dr = d["R"], d["Dr"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    w = torch.randn(H, N + 5, R, generator=g, device="cuda").to(torch.bfloat16)[:, 5:]
    start = torch.zeros(len(keys) + 1, dtype=torch.int32)
    start[1:] = torch.tensor(keys).cumsum(0)
    n = max(1, int(start[-1]) + pad)
    guard = Guarded()
    kv = guard.alloc("kv", n * H * N, torch.bfloat16).view(n, H, N).fill_(5.0)
    kr = guard.alloc("k_rope", n * (Dr + 8), torch.bfloat16).view(n, Dr + 8).fill_(5.0)
    ws = bd.alloc_workspace(256)
    bd.mtp_latent_expand(bd.make_latent_cache(d["pages"], d["table"], Dr), (start if key_start is None else key_start).cuda(), w,
                         kv, kr[:, :Dr], ws)
    torch.cuda.synchronize()
    guard.check()
    assert bd.get_status(ws) == expect
    return w, start.tolist(), kv, kr


def check_expanded(d, keys, H, N, **kw):
    w, start, kv, kr = expanded(d, keys, H, N, **kw)
    R, Dr = d["R"], d["Dr"]
    for b, n in enumerate(keys):
        e, row = slice(start[b], start[b + 1]), d["seqs"][b][:n]
        check_product(row[:, None, :R].expand(-1, H, -1), w, kv[e])
        assert torch.equal(kr[e, :Dr].cpu(), row[:, R:])
    assert (kv[start[-1]:] == 5).all() and (kr[start[-1]:] == 5).all() and (kr[:, Dr:] == 5).all()


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("R,Dr", [(256, 32), (512, 64)])
def test_expand(page, R, Dr):
    total = [1, 129, 0, 300, page]
    d = make_latent([1, 129, 0, 300, page], [0] * 5, 1, R, Dr, page, seed=page)
    check_expanded(d, total, 3, 256, pad=2)
    check_expanded(d, [0, 128, 0, 33, 1], 5, 136)          # not all that the cache holds


def test_expand_sizes_of_heads():
    d = make_latent([70, 200], [0, 0], 1, 512, 64, 64, seed=9)
    for H, N in ((1, 8), (128, 256), (16, 192), (2, 1000)):
        check_expanded(d, [70, 200], H, N)


@pytest.mark.parametrize("R,Dr", [(256, 64), (512, 32)])
def test_expand_of_many_row_tiles(R, Dr):
    """More tiles of rows than there are SMs: rows are kept, given up and brought again."""
    n = [45000, 1, 0, 1300]
    check_expanded(make_latent(n, [0] * 4, 1, R, Dr, 128, seed=R), n, 3, 64, pad=1)


def test_expand_of_many_sequences():
    n = [(b * 5) % 9 for b in range(700)]
    check_expanded(make_latent(n, [0] * 700, 1, 256, 32, 16, seed=1), n, 2, 64, pad=3)


def test_expand_flags():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_latent([40, 60], [0, 0], 1, 256, 64, 16, seed=2)
    d["pages"].nan_to_num_(0.0)
    start = lambda *x: torch.tensor(x, dtype=torch.int32)  # noqa: E731
    _, _, kv, _ = expanded(d, [40, 60], 2, 64, key_start=start(0, 40, 20), expect=bd.STATUS_BAD_ROWS)
    assert (kv[40:] == 5).all()
    _, _, kv, _ = expanded(d, [40, 60], 2, 64, key_start=start(-3, 40, 4000), expect=bd.STATUS_BAD_ROWS)
    _, _, kv, _ = expanded(d, [40, 90], 2, 64, expect=bd.STATUS_BAD_CTX)      # 64 positions of pages
    assert (kv[104:] == 5).all()
    d["table"][1, 1] = 99
    expanded(d, [40, 60], 2, 64, expect=bd.STATUS_BAD_PAGE)


# ------------------------------------------------------------- absorbed attention


@pytest.mark.parametrize("H", [1, 3, 16, 40, 64, 72, 128])
@pytest.mark.parametrize("R,Dr", [(256, 32), (512, 64)])
def test_attend_heads(H, R, Dr):
    d = make_latent([4, 0, 1, 7], [300, 9, 0, 130], H, R, Dr, 64, seed=H, pad=3)
    out, lse = attend(d)
    check_attend(d, out, lse)
    n = sum(d["rows"])
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("R,Dr", [(256, 64), (512, 32)])
def test_attend_pages_and_tile_ends(page, R, Dr):
    rows = [1, 2, 3, 1, 5]
    for ctx in ([126, 127, 128, 254, 250], [0, 1, 15, 16, 63]):
        d = make_latent(rows, ctx, 8, R, Dr, page, seed=page + ctx[0])
        check_attend(d, *attend(d))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 0), (100, 4), (128, 70), (129, 300), (5000, 3)])
@pytest.mark.parametrize("H", [16, 128])
def test_attend_windows(window, sinks, H):
    d = make_latent([3, 1, 20], [700, 5, 260], H, 512, 64, 32, seed=window, window=window, sinks=sinks)
    check_attend(d, *attend(d))
    d = make_latent([2, 40], [0, 300], H, 256, 32, 16, seed=sinks, window=window, sinks=sinks)
    check_attend(d, *attend(d))


@pytest.mark.parametrize("H,rows,ctx", [(16, 70, 0), (16, 333, 150), (128, 40, 100), (40, 129, 1000), (1, 600, 3), (5, 300, 0)])
def test_attend_chunks(H, rows, ctx):
    d = make_latent([rows, 2], [ctx, 500], H, 512, 64, 64, seed=rows)
    check_attend(d, *attend(d))


def test_attend_many_blocks_under_a_window():
    """Every block begins with a tile of four visible keys, so that its maximum grows later."""
    d = make_latent([150, 90, 120], [6000, 600, 3000], 40, 256, 32, 32, seed=1, window=1500, sinks=4)
    check_attend(d, *attend(d))


def test_attend_long_contexts_split_and_joined():
    d = make_latent([2, 1], [6000, 9000], 16, 512, 64, 64, seed=1)
    check_attend(d, *attend(d))
    d = make_latent([1], [20000], 128, 256, 64, 128, seed=2)
    check_attend(d, *attend(d))


@pytest.mark.parametrize("H,rows", [(16, [1] * 20), (128, [1, 0, 2, 1]), (40, [4, 4, 4, 0, 1]), (64, [2] * 9)])
def test_attend_few_items(H, rows):
    """Calls small enough that every CTA makes the plan for itself; and rows that end early."""
    for R, Dr in ((512, 64), (256, 32)):
        d = make_latent(rows, [(b * 531) % 1500 for b in range(len(rows))], H, R, Dr, 32, seed=H, pad=1)
        out, lse = attend(d)
        check_attend(d, out, lse)
        assert (out[sum(rows):] == 7).all()


@pytest.mark.parametrize("n", [12, 17])                       # the plan in every CTA, and in a kernel of its own
def test_attend_one_long_and_many_short(n):
    """Shares of 17 and more items: one sequence is as long as many others are short."""
    long, H = 260000, 128
    d = make_latent([1] * n + [2] + [1] * n, [b % 5 for b in range(n)] + [long] + [b % 7 for b in range(n)], H, 512, 64, 128, seed=3)
    out, lse = attend(d)
    assert torch.isfinite(out).all()
    short = dict(d, rows=[1] * n, ctx=d["ctx"][:n], seqs=d["seqs"][:n], q=d["q"][:n], n_rows=n)
    check_attend(short, out[:n], lse[:n])
    short = dict(d, rows=[1] * n, ctx=d["ctx"][n + 1:], seqs=d["seqs"][n + 1:], q=d["q"][n + 2:], n_rows=n)
    check_attend(short, out[n + 2:], lse[n + 2:])
    k = d["seqs"][n][:, None]
    ref = [x.cpu() for x in attention(d["q"][n:n + 2], k, k[..., :512], sees(long, 2, long + 2, 0, 0).cuda(), d["scale"], "cuda")]
    check_rows(ref, out[n:n + 2], lse[n:n + 2], 2, long + 2)


@pytest.mark.parametrize("B", [64, 600, 1100])
def test_attend_large_batches(B):
    rows = [(b * 7) % 4 for b in range(B)]
    ctx = [(b * 37) % 91 for b in range(B)]
    rows[0] = rows[1] = rows[-1] = rows[-2] = 0
    rows[B // 2] = 60
    d = make_latent(rows, ctx, 8, 256, 32, 16, seed=B, pad=3)
    out, lse = attend(d)
    check_attend(d, out, lse)
    assert (out[sum(rows):] == 7).all()


def test_attend_strided_rows():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_latent([3, 2], [50, 200], 8, 256, 64, 32, seed=4)
    n, H, R = d["n_rows"], 8, 256
    wide = torch.full((n, H * (R + 64) + 40), 3.0, device="cuda", dtype=torch.bfloat16)
    q = wide[:, 16:16 + H * (R + 64)].view(n, H, R + 64)
    q.copy_(d["q"])
    d["q"] = q
    big = torch.full((n, H * R + 24), 5.0, device="cuda", dtype=torch.bfloat16)
    out = big[:, 8:8 + H * R].view(n, H, R)
    ws = bd.alloc_workspace(bd.latent_attn_workspace_size(2, n, H, R))
    bd.mtp_latent_attn(bd.make_latent_cache(d["pages"], d["table"], 64), d["row_start"], d["ctx_len"], q, out, None, ws, d["scale"])
    torch.cuda.synchronize()
    check_attend(d, out, None)
    assert (big[:, :8] == 5).all() and (big[:, 8 + H * R:] == 5).all()


def test_attend_is_the_same_bit_for_bit():
    d = make_latent([4, 4, 90], [3000, 700, 100], 40, 512, 64, 64, seed=8)
    a = [x.clone() for x in attend(d)]
    b = attend(d)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


# ------------------------------------------------------------- expanded attention


@pytest.mark.parametrize("H", [1, 5, 16, 128])
@pytest.mark.parametrize("Dn,Dr,Dv", [(128, 64, 128), (64, 32, 64), (128, 32, 64), (64, 64, 128)])
def test_prefill_heads(H, Dn, Dr, Dv):
    d = make_prompt([4, 0, 130, 7], [30, 9, 0, 200], H, Dn, Dr, Dv, seed=H, pad=3)
    out, lse = prefill(d)
    check_prefill(d, out, lse)
    n = sum(d["rows"])
    assert (out[n:] == 7).all() and (lse[n:] == 7).all()


@pytest.mark.parametrize("rows,ctx", [([1], [0]), ([127, 128, 129], [0, 0, 0]), ([255, 256, 257], [1, 128, 127]), ([700], [500]),
                                      ([1, 1, 1], [126, 127, 128])])
def test_prefill_tile_ends(rows, ctx):
    d = make_prompt(rows, ctx, 3, 128, 64, 128, seed=rows[0], key_pad=5)
    check_prefill(d, *prefill(d))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (64, 0), (100, 4), (129, 300), (5000, 3)])
def test_prefill_windows(window, sinks):
    d = make_prompt([3, 1, 320], [700, 5, 260], 4, 128, 64, 128, seed=window, window=window, sinks=sinks)
    check_prefill(d, *prefill(d))


def test_prefill_long_context_split_and_joined():
    d = make_prompt([2, 40], [6000, 4000], 2, 128, 64, 128, seed=1)
    check_prefill(d, *prefill(d))


@pytest.mark.parametrize("B", [64, 600, 1100])
def test_prefill_large_batches(B):
    rows = [(b * 7) % 4 for b in range(B)]
    ctx = [(b * 37) % 91 for b in range(B)]
    rows[0] = rows[1] = rows[-1] = rows[-2] = 0
    rows[B // 2] = 300
    d = make_prompt(rows, ctx, 2, 64, 32, 64, seed=B, pad=3)
    check_prefill(d, *prefill(d))


def test_prefill_few_items():
    for rows, ctx, H in (([1, 2, 0, 1], [900, 5, 7, 0], 8), ([300], [40], 4), ([1], [0], 1), ([257, 3], [1000, 2000], 16)):
        d = make_prompt(rows, ctx, H, 128, 64, 128, seed=H, pad=1)
        check_prefill(d, *prefill(d))


def test_prefill_of_fresh_prompts_takes_row_start():
    d = make_prompt([9, 300, 0, 41], [0] * 4, 4, 128, 64, 128, seed=3)
    check_prefill(d, *prefill(d, key_start=d["row_start"]))


def test_prefill_is_the_same_bit_for_bit():
    d = make_prompt([4, 300, 90], [3000, 700, 100], 8, 128, 64, 128, seed=8)
    a = [x.clone() for x in prefill(d)]
    b = prefill(d)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
