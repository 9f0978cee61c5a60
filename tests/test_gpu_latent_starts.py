"""mtp_latent_expand of starts that decrease: rows would be counted twice, so that nothing
of the call is written."""

import pytest
import torch

from latent_helpers import check_product, make_latent

pytestmark = pytest.mark.gpu


def expand(d, start, n, H=2, N=64):
    """(w, kv, k_rope, status) of the starts over n rows between guard bands."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    from mtp_speculative_decoding_draft_gb300.model import Guarded
    w = torch.randn(H, N, d["R"], generator=torch.Generator(device="cuda").manual_seed(3), device="cuda").to(torch.bfloat16)
    guard = Guarded()
    kv = guard.alloc("kv", n * H * N, torch.bfloat16).view(n, H, N).fill_(5.0)
    kr = guard.alloc("k_rope", n * d["Dr"], torch.bfloat16).view(n, d["Dr"]).fill_(5.0)
    ws = bd.alloc_workspace(256)
    bd.mtp_latent_expand(bd.make_latent_cache(d["pages"], d["table"], d["Dr"]),
                         torch.tensor(start, dtype=torch.int32, device="cuda"), w, kv, kr, ws)
    torch.cuda.synchronize()
    guard.check()
    return w, kv, kr, bd.get_status(ws)


@pytest.mark.parametrize("start", [(0, 40, 20, 60), (0, 60, 0, 60), (0, 1, 0, 0), (0, 40, -20, 60), (-8, -9, 40, 60),
                                   (0, 40, 60, 59), (0, 40, 20, 4000)])
def test_starts_that_decrease_write_nothing(start):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_latent([60, 60, 60], [0, 0, 0], 1, 256, 64, 16, seed=2)
    for n in (60, 300):                                        # one tile of rows, and pairs of CTAs
        _, kv, kr, status = expand(d, start, n)
        assert status == bd.STATUS_BAD_ROWS
        assert (kv == 5).all() and (kr == 5).all()


@pytest.mark.parametrize("B", [4, 600, 4001])
def test_many_starts_that_alternate_write_nothing(B):
    """Summed up, these starts have far more row tiles than the rows, and than the table, have."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_latent([1] * B, [0] * B, 1, 256, 32, 16, seed=4)
    d["table"] = torch.zeros(B, 1024, dtype=torch.int32, device="cuda")
    d["pages"].zero_()
    _, kv, kr, status = expand(d, [0, 16384] * (B // 2) + [0] * (B % 2 + 1), 16384)
    assert status == bd.STATUS_BAD_ROWS
    assert (kv == 5).all() and (kr == 5).all()


@pytest.mark.parametrize("start", [(-3, 40, 60, 90), (0, 40, 60, 4000), (-9, -5, 20, 60)])
def test_starts_outside_the_rows_drop_their_sequence_alone(start):
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    d = make_latent([60, 60, 60], [0, 0, 0], 1, 256, 64, 16, seed=2)
    w, kv, kr, status = expand(d, start, 90)
    assert status == bd.STATUS_BAD_ROWS
    left = torch.ones(90, dtype=torch.bool, device="cuda")
    for b, (s, e) in enumerate(zip(start, start[1:])):
        if s < 0 or e > 90:
            continue
        left[s:e] = False
        row = d["seqs"][b][:e - s]
        check_product(row[:, None, :256].expand(-1, 2, -1), w, kv[s:e])
        assert torch.equal(kr[s:e].cpu(), row[:, 256:])
    assert (kv[left] == 5).all() and (kr[left] == 5).all()
