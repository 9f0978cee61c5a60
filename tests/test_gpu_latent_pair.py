"""Absorbed attention on pairs of CTAs: what the second CTA hands over to the products that
the first one issues."""

import pytest
import torch

from latent_helpers import attend, check_attend, make_latent

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("R,Dr", [(512, 64), (256, 32)])
def test_weights_and_rescaled_sums_are_there_in_time(R, Dr):
    """Maxima that grow from tile to tile, so that every tile rescales the sums before the product
    with its weights; items of many tiles, and of few.  Weights or sums that were read
    too early would differ between the runs."""
    d = make_latent([6, 4, 9, 4, 2, 30], [3000, 40, 1500, 700, 5000, 260], 64, R, Dr, 64, seed=R)
    for b, k in enumerate(d["seqs"]):
        k *= torch.linspace(0.1, 8.0, k.shape[0])[:, None]
        j = torch.arange(k.shape[0])
        d["pages"][d["table"][b, j // 64].long(), j % 64] = k.cuda()
    d["q"] *= 4
    out, lse = (x.clone() for x in attend(d))
    check_attend(d, out, lse)
    for _ in range(60):
        o, z = attend(d)
        assert torch.equal(o, out) and torch.equal(z, lse)
