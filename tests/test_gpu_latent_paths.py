"""Paths of the latent-attention kernels that sizes near the usual ones do not take: row tiles past
those that a CTA keeps places of, odd products on pairs of CTAs, pairs with the other rotary size."""

import pytest

from latent_helpers import attend, check_attend, make_latent
from test_gpu_latent import check_expanded, product

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,R,Dr", [([12288 - 77 * b for b in range(16)], 256, 32),          # 1464 tiles of a few long contexts
                                    ([(b * 37) % 401 for b in range(900)], 256, 64),         # 1782 of three sequences a thread
                                    ([1] * 1100 + [0, 300, 129], 512, 64)])                  # past the place 1024 by a sequence each
def test_expand_past_the_tiles_whose_places_are_kept(n, R, Dr):
    assert sum((x + 127) // 128 for x in n) > 1024
    check_expanded(make_latent(n, [0] * len(n), 1, R, Dr, 128, seed=len(n)), n, 2, 24, pad=3)


@pytest.mark.parametrize("n", [129, 391])
@pytest.mark.parametrize("K,N", [(8, 8), (40, 24), (72, 136), (200, 1000), (1032, 264)])
@pytest.mark.parametrize("transposed", [True, False])
@pytest.mark.parametrize("order", ["rows", "heads"])
def test_products_of_odd_sizes_on_pairs(n, K, N, transposed, order):
    product(n, 3, K, N, transposed, seed=K, order=order)


def test_products_of_odd_sizes_and_many_heads_on_pairs():
    product(300, 90, 72, 136, True, order="heads")
    product(140, 128, 40, 264, False, order="heads")


@pytest.mark.parametrize("R,Dr", [(512, 32), (512, 64), (256, 64), (256, 32)])
@pytest.mark.parametrize("H,rows,ctx", [(128, [4, 1, 9], [300, 0, 2000]), (40, [130, 3], [70, 900]), (3, [300], [500])])
def test_attend_on_pairs_with_either_rotary_size(R, Dr, H, rows, ctx):
    assert -(-sum(rows) // len(rows)) * H > 128
    for page in (16, 128):
        d = make_latent(rows, ctx, H, R, Dr, page, seed=H + R, pad=2)
        out, lse = attend(d)
        check_attend(d, out, lse)
        assert (out[sum(rows):] == 7).all()
    d = make_latent(rows, ctx, H, R, Dr, 32, seed=H + R, window=100, sinks=3)
    check_attend(d, *attend(d))
