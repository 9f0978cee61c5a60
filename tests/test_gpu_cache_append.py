"""mtp_cache_append against its definition in 64 bits."""

import pytest
import torch

from paged_helpers import append_reference, make_case

pytestmark = pytest.mark.gpu


def append(d, rot, half=True, scale=1.0, base=10000.0, in_place=False, with_q=True, seed=1, rope=True, expect=0):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    n, Hq, Hkv, Dh, page = d["n_rows"], d["Hq"], d["Hkv"], d["Dh"], d["page"]
    g = torch.Generator(device="cuda").manual_seed(seed)
    qkv = torch.randn(n, (Hq + 2 * Hkv) * Dh, generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = (x.view(n, -1, Dh) for x in qkv.split([Hq * Dh, Hkv * Dh, Hkv * Dh], dim=1))
    q0, k0, v0 = q.clone(), k.clone(), v.clone()
    out = q if in_place else torch.full((n, Hq, Dh), 9.0, device="cuda", dtype=torch.bfloat16)
    cache = bd.make_paged_cache(d["k_pages"], d["v_pages"], d["table"])
    f, _ = bd.rope_frequencies(rot, base)
    r = bd.make_rope(bd.rope_table(f).cuda(), rot, bd.ROPE_HALF if half else bd.ROPE_INTERLEAVED, scale) if rope else None
    before = (d["k_pages"].clone(), d["v_pages"].clone())
    ws = bd.alloc_workspace(256)
    bd.mtp_cache_append(cache, r, d["row_start"], d["ctx_len"], q if with_q else None, k, v, out if with_q else None, ws)
    torch.cuda.synchronize()
    assert bd.get_status(ws) == expect
    return q0, k0, v0, out, before, f


def check(d, rot, half=True, scale=1.0, rope=True, in_place=False, with_q=True, **kw):
    q, k, v, out, (kb, vb), f = append(d, rot, half, scale, rope=rope, in_place=in_place, with_q=with_q, **kw)
    n = sum(d["rows"])
    pos = torch.cat([torch.arange(c, c + r) for c, r in zip(d["ctx"], d["rows"])])
    seq = torch.cat([torch.full((r,), b) for b, r in enumerate(d["rows"])]).long()
    if not rope:
        f, scale = torch.zeros_like(f), 1.0

    def near(got, x):
        ref, mag = append_reference(x[:n], pos, f, rot, half, scale)
        # rounded to bf16 (2^-8); sine and cosine of an angle off by 2^-25 of a
        # half turn, good to 2 ulp, the two products and their sum: 2^-20 in all
        tol = 2.0 ** -8 * ref.abs() + 2.0 ** -20 * mag
        err = (got.double().cpu() - ref).abs()
        assert (err <= tol).all(), float((err / tol.clamp(min=1e-30)).max())

    if with_q:
        near(out[:n], q)
        assert torch.equal(out[n:], q[n:] if in_place else torch.full_like(out[n:], 9.0))
    page = d["table"].cpu()[seq, pos // d["page"]].long()
    slot = pos % d["page"]
    near(d["k_pages"].cpu()[page, :, slot], k)
    assert torch.equal(d["v_pages"].cpu()[page, :, slot], v[:n].cpu())
    # every other slot is as it was
    for now, was in ((d["k_pages"], kb), (d["v_pages"], vb)):
        now, was = now.cpu().clone(), was.cpu().clone()
        now[page, :, slot] = 0
        was[page, :, slot] = 0
        assert torch.equal(now.view(torch.int16), was.view(torch.int16))


@pytest.mark.parametrize("Hq,Hkv,Dh", [(2, 2, 32), (14, 2, 64), (32, 8, 128), (40, 8, 128)])
@pytest.mark.parametrize("half", [True, False])
@pytest.mark.parametrize("part", [1, 2, 4])
def test_layouts_and_partial_heads(Hq, Hkv, Dh, half, part):
    check(make_case([1, 0, 5, 3], [0, 7, 62, 300], Hq, Hkv, Dh, 64, seed=part, pad=2), Dh // part, half, 1.2)


@pytest.mark.parametrize("page", [16, 32, 64, 128])
def test_pages(page):
    check(make_case([40, 1, 17], [page - 1, page, 3 * page + 5], 8, 2, 64, page, seed=page), 64)


@pytest.mark.parametrize("rot", [8, 24, 40, 48, 56])
@pytest.mark.parametrize("half", [True, False])
def test_odd_rotated_parts(rot, half):
    check(make_case([3, 2], [11, 90], 6, 2, 64, 32, seed=rot), rot, half)


def test_far_positions():
    """At position 10^6 an fp32 angle would be off by 0.06."""
    d = make_case([4], [60], 4, 2, 32, 64, seed=4)
    far = 1_000_003
    width = (far + 4 + 63) // 64
    table = torch.full((1, width), -1, dtype=torch.int32, device="cuda")
    table[0, -1], table[0, -2] = 0, 1
    d.update(table=table, ctx=[far])
    d["ctx_len"].fill_(far)
    check(d, 32)


def test_many_rows_and_sequences():
    rows = [(i * 5) % 7 for i in range(900)]
    check(make_case(rows, [(i * 13) % 50 for i in range(900)], 2, 1, 32, 16, seed=2, pad=4), 32)


def test_in_place_keys_only_and_no_rotation():
    check(make_case([2, 6], [5, 100], 8, 2, 128, 64, seed=1), 128, in_place=True)
    check(make_case([2, 6], [5, 100], 8, 2, 128, 64, seed=1), 128, with_q=False)
    check(make_case([2, 6], [5, 100], 8, 2, 128, 64, seed=1), 128, rope=False)


def test_device_side_errors_drop_the_row():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_case([4], [62], 4, 2, 64, 64, seed=3)
    d["table"][0, 1] = 1000
    _, _, _, _, (kb, _), _ = append(d, 64, expect=bd.STATUS_BAD_PAGE)
    page = int(d["table"][0, 0])
    same = (d["k_pages"].view(torch.int16) == kb.view(torch.int16)).all(-1).all(1)
    assert same.sum() == same.numel() - 2 and not same[page, 62] and not same[page, 63]
    d["ctx_len"].fill_(1 << 25)
    _, _, _, _, (kb, _), _ = append(d, 64, expect=bd.STATUS_BAD_CTX)
    assert torch.equal(d["k_pages"].view(torch.int16), kb.view(torch.int16))
    d["ctx_len"].fill_(0)
    d["row_start"].copy_(torch.tensor([2, 400], dtype=torch.int32))
    append(d, 64, expect=bd.STATUS_BAD_ROWS)
