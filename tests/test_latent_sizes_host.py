"""Workspace sizes of the latent-attention operators: a workspace for a largest batch serves
every smaller one.  No GPU needed."""

import ctypes
import random

import pytest

from mtp_speculative_decoding_draft_gb300 import binding as bd
from mtp_speculative_decoding_draft_gb300 import build


@pytest.fixture(scope="module")
def sizes():
    build.build()
    return {"attn": bd.latent_attn_workspace_size, "prefill": bd.latent_prefill_workspace_size}


def test_sequences_that_finish_need_no_larger_workspace(sizes):
    """The mean number of rows a sequence, and with it the kernel, differs on the two sides."""
    attn = sizes["attn"]
    for big, small in (((64, 256, 16, 256), (24, 256, 16, 256)), ((1024, 4096, 16, 512), (64, 4096, 16, 512)),
                       ((64, 256, 16, 256), (64, 64, 16, 256)), ((8, 8, 128, 256), (1, 8, 128, 256))):
        assert attn(*small) <= attn(*big)


@pytest.mark.parametrize("kind,D", [("attn", 256), ("attn", 512), ("prefill", 64), ("prefill", 128)])
def test_sizes_grow_with_sequences_and_rows(sizes, kind, D):
    rnd = random.Random(D)
    for _ in range(4000):
        B, n, H = int(2 ** rnd.uniform(0, 20)), int(2 ** rnd.uniform(0, 29)), rnd.randint(1, 128)
        b, m = rnd.choice([1, B, rnd.randint(1, B)]), rnd.choice([1, n, rnd.randint(1, n)])
        assert 256 < sizes[kind](b, m, H, D) <= sizes[kind](B, n, H, D), (b, m, B, n, H)


def test_small_calls_take_the_small_states(sizes):
    """A call that no pair of CTAs serves does not ask for the pairs' states."""
    assert sizes["attn"](8, 8, 16, 256) < 22 << 20 < sizes["attn"](8, 16, 16, 256)


OK, OTHER, THIRD = (ctypes.c_void_p(1 << i) for i in (20, 21, 22))      # aligned, never read
WORKSPACE = -3
ITEM = 48                                                               # bytes of an item of the plan


@pytest.mark.parametrize("H", [1, 39, 64, 65, 127, 128])
def test_the_largest_calls_are_counted_in_31_bits(sizes, H):
    """At the largest numbers of sequences and rows there is a workspace size, of fewer than 2^31
    items, and a call without the workspace is refused for that alone."""
    B, n = 1 << 20, 1 << 29
    lib = bd.library()
    for R in (256, 512):
        size = sizes["attn"](B, n, H, R)
        # 2 r (n / t + B) items of the first choice of blocks, r runs of t tokens, R / 256 items each
        items = 2 * (R // 256) * (n // (2 * (128 // H)) + B)
        assert items * ITEM <= size < items * ITEM + (1 << 27) and items < 1 << 31
        cache = bd.MtpLatentCache(R, 64, 64, 100, 10, OK, OK)
        call = lib.mtp_latent_attn(cache, B, H, n, OK, OK, OK, H * (R + 64), 0.1, 0, 0, OTHER, H * R, None, OK, size - 1, None)
        assert call == WORKSPACE
    size, items = sizes["prefill"](B, n, H, 128), (n // 256 + B) * H
    assert items * ITEM <= size < items * ITEM + (1 << 27) and items < 1 << 31
    call = lib.mtp_latent_prefill(B, H, 128, 64, 128, n, 1 << 30, OK, OK, OK, OK, H * 192, THIRD, H * 256, OK, 64, 0.1, 0, 0, OTHER,
                                  H * 128, None, OK, size - 1, None)
    assert call == WORKSPACE
