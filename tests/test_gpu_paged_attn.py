"""mtp_paged_attn against its definition in 64 bits."""

import pytest
import torch

from paged_helpers import check_attend, make_case

pytestmark = pytest.mark.gpu


def attend(d, max_rows=0, scale=0.0, lse=True, q=None, out=None):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    cache = bd.make_paged_cache(d["k_pages"], d["v_pages"], d["table"])
    n, Hq, Dh = d["n_rows"], d["Hq"], d["Dh"]
    q = d["q"] if q is None else q
    out = torch.full((n, Hq, Dh), 7.0, device="cuda", dtype=torch.bfloat16) if out is None else out
    ls = torch.full((n, Hq), 7.0, device="cuda") if lse else None
    ws = bd.alloc_workspace(bd.paged_attn_workspace_size(d["B"], n, max_rows, Hq, d["Hkv"], Dh))
    bd.mtp_paged_attn(cache, d["row_start"], d["ctx_len"], q, out, ls, ws, scale=scale, window=d["window"],
                      sinks=d["sinks"], max_rows=max_rows)
    torch.cuda.synchronize()
    return out, ls, bd.get_status(ws)


def run(d, **kw):
    out, lse, status = attend(d, **kw)
    assert status == 0
    check_attend(d, out, lse, kw.get("scale") or None)
    n = sum(d["rows"])
    assert (out[n:] == 7.0).all() and (lse is None or (lse[n:] == 7.0).all())   # padding is left alone
    return out, lse


@pytest.mark.parametrize("Hq,Hkv,Dh", [(2, 2, 32), (8, 2, 32), (8, 8, 64), (14, 2, 64), (32, 8, 128), (40, 8, 128), (8, 1, 128)])
@pytest.mark.parametrize("page", [16, 128])
def test_decode_and_verify_rows(Hq, Hkv, Dh, page):
    run(make_case([1, 4, 0, 9, 2], [0, 63, 5, 300, 128], Hq, Hkv, Dh, page, seed=Hq + page, pad=3))


@pytest.mark.parametrize("page", [16, 32, 64, 128])
@pytest.mark.parametrize("ctx", [0, 1, 15, 16, 60, 61, 63, 64, 65, 127, 128, 129])
def test_lengths_around_pages_and_tiles(page, ctx):
    run(make_case([4], [ctx], 8, 2, 64, page, seed=ctx))


@pytest.mark.parametrize("rows", [1, 2, 4, 5, 8, 9, 16, 17, 33])
@pytest.mark.parametrize("Hq,Hkv,Dh", [(32, 8, 128), (10, 2, 64)])
def test_row_counts(rows, Hq, Hkv, Dh):
    run(make_case([rows], [197], Hq, Hkv, Dh, 32, seed=rows), max_rows=rows)


@pytest.mark.parametrize("rows,ctx", [([70], [0]), ([257], [100]), ([64, 1, 300, 0, 3], [7, 500, 0, 3, 64]), ([130, 515], [1000, 129])])
@pytest.mark.parametrize("Hq,Hkv,Dh,page", [(8, 2, 128, 64), (10, 2, 128, 16), (4, 4, 64, 32), (6, 2, 64, 128), (3, 1, 32, 16), (7, 1, 128, 64)])
def test_chunks_of_prompts(rows, ctx, Hq, Hkv, Dh, page):
    run(make_case(rows, ctx, Hq, Hkv, Dh, page, seed=len(rows) + rows[0], pad=2))


@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 4), (7, 0), (64, 3), (100, 70), (1000, 4), (129, 128), (5, 500)])
@pytest.mark.parametrize("rows,ctx", [([4, 1], [300, 17]), ([150, 3], [700, 0]), ([2, 90], [5, 64])])
@pytest.mark.parametrize("Dh", [64, 128])
def test_window_and_sinks(window, sinks, rows, ctx, Dh):
    run(make_case(rows, ctx, 8, 2, Dh, 32, seed=window, window=window, sinks=sinks))


@pytest.mark.parametrize("Dh,rows", [(128, 4), (64, 2), (32, 4), (128, 90)])
def test_long_context_is_split_and_joined(Dh, rows):
    run(make_case([rows], [9000], 4, 1, Dh, 64, seed=Dh))


def test_many_sequences():
    rows = [(i * 7) % 6 for i in range(333)]
    ctx = [(i * 37) % 211 for i in range(333)]
    run(make_case(rows, ctx, 4, 2, 64, 16, seed=3, pad=1), max_rows=5)


@pytest.mark.parametrize("hint", [0, 1, 3, 40, 10000])
def test_the_hint_chooses_a_kernel_only(hint):
    run(make_case([3, 40, 1], [100, 20, 300], 8, 2, 128, 64, seed=8), max_rows=hint)


def test_scale_strides_and_no_lse():
    d = make_case([3, 80], [50, 130], 8, 2, 128, 64, seed=5)
    wide = torch.zeros(d["n_rows"], 8 * 128 + 64, device="cuda", dtype=torch.bfloat16)
    wide[:, 32:32 + 1024] = d["q"].flatten(1)
    q = wide[:, 32:32 + 1024].view(d["n_rows"], 8, 128)
    room = torch.full((d["n_rows"], 1024 + 8), 3.0, device="cuda", dtype=torch.bfloat16)
    out = room[:, :1024].view(d["n_rows"], 8, 128)
    run(d, scale=0.2, lse=False, q=q, out=out)
    assert (room[:, 1024:] == 3.0).all()


def test_large_scores_and_equal_scores():
    d = make_case([4, 70], [200, 60], 8, 2, 128, 64, seed=6)
    run(d, scale=3.0)        # weights concentrate on single keys
    run(d, scale=1e-6)       # weights all alike


def test_rows_repeat_bit_for_bit():
    d = make_case([4, 130, 1], [3000, 700, 5000], 8, 2, 128, 64, seed=9)
    a, la, _ = attend(d)
    for _ in range(3):
        b, lb, _ = attend(d)
        assert torch.equal(a, b) and torch.equal(la, lb)


def test_a_graph_replays_on_new_inputs_and_another_stream():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_case([4, 90], [500, 64], 8, 2, 128, 64, seed=10)
    cache = bd.make_paged_cache(d["k_pages"], d["v_pages"], d["table"])
    out, lse = torch.zeros_like(d["q"]), torch.zeros(d["n_rows"], 8, device="cuda")
    ws = bd.alloc_workspace(bd.paged_attn_workspace_size(2, d["n_rows"], 0, 8, 2, 128))
    call = lambda: bd.mtp_paged_attn(cache, d["row_start"], d["ctx_len"], d["q"], out, lse, ws)  # noqa: E731
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        call()
    side.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    d["q"].copy_(torch.randn_like(d["q"]))
    g.replay()
    torch.cuda.synchronize()
    check_attend(d, out, lse)
    # other lengths of the same arrays
    d["ctx_len"].copy_(torch.tensor([100, 0], dtype=torch.int32))
    g.replay()
    torch.cuda.synchronize()
    d["ctx"] = [100, 0]
    d["seqs"] = [(k[:c + r], v[:c + r]) for (k, v), c, r in zip(d["seqs"], d["ctx"], d["rows"])]
    check_attend(d, out, lse)
    assert bd.get_status(ws) == 0


def test_device_side_errors_are_flagged_and_bounded():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_case([4], [60], 8, 2, 64, 64, seed=11)
    d["k_pages"].nan_to_num_(0.0)
    d["v_pages"].nan_to_num_(0.0)
    d["ctx_len"].fill_(10 ** 6)                                   # past the cache
    assert attend(d)[2] == bd.STATUS_BAD_CTX
    d["ctx_len"].fill_(-3)
    assert attend(d)[2] == bd.STATUS_BAD_CTX
    d["ctx_len"].fill_(60)
    d["row_start"].copy_(torch.tensor([0, 1000], dtype=torch.int32))
    assert attend(d)[2] & bd.STATUS_BAD_ROWS
    d["row_start"].copy_(torch.tensor([3, 0], dtype=torch.int32))
    out, lse, st = attend(d)
    assert st == bd.STATUS_BAD_ROWS and (out == 7.0).all()
    d["row_start"].copy_(torch.tensor([0, 4], dtype=torch.int32))
    d["table"][0, 0] = 1 << 20
    assert attend(d)[2] == bd.STATUS_BAD_PAGE


@pytest.mark.parametrize("rows", [3, 80])
def test_a_row_that_sees_nothing_is_zero(rows):
    """A context past the cache puts the window's keys outside it: no key is left."""
    d = make_case([rows], [64 - rows % 64], 4, 2, 64, 64, seed=12, spare=0)
    d["k_pages"].nan_to_num_(0.0)
    d["v_pages"].nan_to_num_(0.0)
    d["ctx_len"].fill_(10 ** 6)
    d["window"] = 1
    out, lse, st = attend(d)
    assert st & 4
    assert (out[:rows] == 0).all() and torch.isneginf(lse[:rows]).all()


@pytest.mark.parametrize("rows", [4, 70])
def test_a_pool_past_32_bits(rows):
    """Elements past 2^32: 8.6 GB pools whose last pages hold the sequence."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_case([rows], [200], 8, 2, 128, 128, seed=13)
    n_pages = 2 ** 32 // (2 * 128 * 128) + 7
    big = [torch.empty(n_pages, 2, 128, 128, device="cuda", dtype=torch.bfloat16) for _ in range(2)]
    table = torch.zeros_like(d["table"])
    for i in range(table.shape[1]):
        table[0, i] = n_pages - 1 - i
        for pool, name in zip(big, ("k_pages", "v_pages")):
            pool[n_pages - 1 - i] = d[name][int(d["table"][0, i])]
    # the last rows come through the append
    ws = bd.alloc_workspace(256)
    k, v = (x[200:].cuda() for x in d["seqs"][0])
    for pool in big:
        for j in range(200, 200 + rows):
            pool[n_pages - 1 - j // 128, :, j % 128] = float("nan")
    bd.mtp_cache_append(bd.make_paged_cache(big[0], big[1], table), None, d["row_start"], d["ctx_len"], None, k, v, None, ws)
    d.update(k_pages=big[0], v_pages=big[1], table=table)
    run(d)
    assert bd.get_status(ws) == 0


def test_two_streams_with_workspaces_of_their_own():
    cases = [make_case([4] * 20, [900 + 37 * i for i in range(20)], 8, 2, 128, 64, seed=14),
             make_case([90, 4, 200], [700, 30, 400], 8, 2, 128, 64, seed=15),
             make_case([2] * 9, [2000 + i for i in range(9)], 8, 2, 64, 16, seed=16, window=500, sinks=4)]
    alone = [attend(d)[:2] for d in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    for turn in range(4):
        got = []
        for d, s in zip(cases, streams):
            s.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(s):
                from mtp_speculative_decoding_draft_gb300 import binding as bd
                cache = bd.make_paged_cache(d["k_pages"], d["v_pages"], d["table"])
                out, lse = torch.full_like(d["q"], 7.0), torch.full((d["n_rows"], d["Hq"]), 7.0, device="cuda")
                ws = bd.alloc_workspace(bd.paged_attn_workspace_size(d["B"], d["n_rows"], 0, d["Hq"], d["Hkv"], d["Dh"]))
                for _ in range(3):
                    bd.mtp_paged_attn(cache, d["row_start"], d["ctx_len"], d["q"], out, lse, ws, window=d["window"], sinks=d["sinks"])
                got.append((out, lse, ws))
        torch.cuda.synchronize()
        for (o, l, _), (ro, rl) in zip(got, alone):
            assert torch.equal(o, ro) and torch.equal(l, rl)


def test_calls_of_many_shapes_share_a_workspace():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    cases = [make_case([90, 4, 200], [700, 30, 400], 8, 2, 128, 64, seed=15), make_case([1], [5000], 8, 2, 128, 64, seed=17),
             make_case([3, 9], [10, 900], 8, 1, 64, 16, seed=18), make_case([40] * 30, [64] * 30, 4, 4, 32, 16, seed=19)]
    ws = bd.alloc_workspace(max(bd.paged_attn_workspace_size(d["B"], d["n_rows"], 0, d["Hq"], d["Hkv"], d["Dh"]) for d in cases))
    for d in cases + cases[::-1]:
        out, lse = torch.full_like(d["q"], 7.0), torch.full((d["n_rows"], d["Hq"]), 7.0, device="cuda")
        bd.mtp_paged_attn(bd.make_paged_cache(d["k_pages"], d["v_pages"], d["table"]), d["row_start"], d["ctx_len"], d["q"], out,
                          lse, ws)
        check_attend(d, out, lse)
    assert bd.get_status(ws) == 0
