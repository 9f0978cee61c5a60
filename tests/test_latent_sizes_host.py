"""Workspace sizes of the latent-attention operators: a workspace for a largest batch serves
every smaller one.  No GPU needed."""

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
