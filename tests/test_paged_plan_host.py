"""Room for the tensor-core kernel's plan: the items that it writes, counted from the
rows on the host, against the workspace that the library asks for.  No GPU needed."""

import random

import pytest

from mtp_speculative_decoding_draft_gb300 import binding as bd
from mtp_speculative_decoding_draft_gb300 import build

CTAS, MAX_CTAS, BLOCK_ROWS = 152, 160, 256


def up256(x):
    return (x + 255) // 256 * 256


def room(B, n_rows, Hq, Hkv, Dh):
    """Items that fit behind the workspace's other parts (status, descriptions, states,
    starts, block counts)."""
    size = bd.paged_attn_workspace_size(B, n_rows, 0, Hq, Hkv, Dh)
    fixed = 256 + up256(MAX_CTAS * 16) + up256(MAX_CTAS * 2 * BLOCK_ROWS * 8) + up256(MAX_CTAS * 2 * BLOCK_ROWS * Dh * 4)
    return (size - fixed - up256(MAX_CTAS * 80) - up256(4 * (B + 1))) // 48


def places(row_start, n_rows, G, Hkv, ordered_only=True):
    """Items written: every sequence's blocks on every K/V head, and the gaps of the last round."""
    if ordered_only and any(e < a for a, e in zip(row_start, row_start[1:])):
        return 0
    tpb, items = 2 * (128 // G), 0
    for a, e in zip(row_start, row_start[1:]):
        first = min(max(a, 0), n_rows)
        n = min(max(e, first), n_rows) - first
        items += (n + tpb - 1) // tpb * Hkv
    return (items + CTAS - 1) // CTAS * CTAS


@pytest.fixture(scope="module", autouse=True)
def lib():
    build.build()
    return bd.library()


def test_row_starts_in_order_fit():
    r = random.Random(3)
    for _ in range(3000):
        B, n, G, Hkv = r.randint(1, 40), r.randint(70, 5000), r.randint(1, 8), r.randint(1, 16)
        rs = sorted(r.randint(-50, n + 50) for _ in range(B + 1))
        assert places(rs, n, G, Hkv) <= room(B, n, G * Hkv, Hkv, 128), (rs, n, G, Hkv)


@pytest.mark.parametrize("B,rs", [(4, [0, 4096, 0, 4096, 0]), (64, [0, 4096] * 32 + [0])])
def test_row_starts_that_decrease_would_not(B, rs):
    """Counted row by row they need more than there is: the plan takes no item of them."""
    assert places(rs, 4096, 4, 8, ordered_only=False) > room(B, 4096, 32, 8, 128)
    assert places(rs, 4096, 4, 8) == 0
