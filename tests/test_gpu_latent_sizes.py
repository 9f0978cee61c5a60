"""One workspace, sized for the largest batch, for every smaller one."""

import pytest
import torch

from latent_helpers import attend, check_attend, check_prefill, make_latent, make_prompt, prefill

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("H,R,Dr", [(16, 256, 32), (16, 512, 64), (40, 256, 64), (128, 512, 32)])
def test_a_workspace_of_the_largest_batch_serves_what_is_left_of_it(H, R, Dr):
    """Sequences finish and the same arrays hold fewer of them: other blocks, another kernel."""
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    from mtp_speculative_decoding_draft_gb300.model import Guarded
    guard = Guarded()
    ws = guard.alloc("workspace", bd.latent_attn_workspace_size(64, 256, H, R), torch.uint8)
    for B, each, pad in ((64, 4, 0), (64, 1, 0), (24, 1, 232), (24, 7, 0), (3, 80, 16), (1, 256, 0), (7, 36, 4), (1, 1, 0)):
        d = make_latent([each] * B, [(b * 97) % 700 for b in range(B)], H, R, Dr, 32, seed=B, pad=pad)
        assert d["n_rows"] <= 256
        check_attend(d, *attend(d, ws=ws))
        guard.check()


def test_a_workspace_of_the_largest_prompts_serves_smaller_ones():
    from mtp_speculative_decoding_draft_gb300 import binding as bd
    from mtp_speculative_decoding_draft_gb300.model import Guarded
    guard = Guarded()
    ws = guard.alloc("workspace", bd.latent_prefill_workspace_size(16, 700, 8, 128), torch.uint8)
    for rows in ([40] * 16, [700], [1] * 16, [300, 3, 390]):
        d = make_prompt(rows, [(b * 97) % 500 for b in range(len(rows))], 8, 128, 64, 128, seed=len(rows))
        check_prefill(d, *prefill(d, ws=ws))
        guard.check()
