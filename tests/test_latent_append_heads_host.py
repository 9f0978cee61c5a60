"""Strides of mtp_latent_append's queries, either order.  No GPU needed."""

import ctypes

from mtp_speculative_decoding_draft_gb300 import binding as bd
from mtp_speculative_decoding_draft_gb300 import build

OK, OTHER = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)          # aligned, never read
INVALID, WORKSPACE = -1, -3


def append(n=8, H=32, ldq=192, hsq=8 * 192, ldqo=64, hsqo=8 * 64, qo=OTHER):
    cache = bd.MtpLatentCache(512, 64, 64, 100, 10, OK, OK)
    return bd.library().mtp_latent_append(cache, None, 2, H, n, OK, OK, OK, 576, None, 0.0, OK, ldq, hsq, qo, ldqo, hsqo, OK, 0, None)


def test_heads_of_rows_are_taken():
    build.build()
    assert append() == WORKSPACE                                       # all but the workspace is in order
    assert append(qo=OK, ldqo=192, hsqo=8 * 192) == WORKSPACE          # in place
    assert append(hsq=7 * 192 + 64) == WORKSPACE                       # the last row ends the head
    assert append(n=1, ldq=64, hsq=64, ldqo=64, hsqo=64) == WORKSPACE  # one row: its heads side by side


def test_rows_on_top_of_heads_are_refused():
    build.build()
    for k in ({"hsq": 7 * 192 + 56}, {"hsqo": 7 * 64 + 56}, {"ldq": 64, "hsq": 64}, {"ldq": 56}, {"hsqo": 0}, {"ldqo": -64},
              {"ldq": 1 << 38}, {"hsq": 1 << 38}, {"hsq": 8 * 192 + 4}):
        assert append(**k) == INVALID, k
    assert append(n=1 << 29, ldq=1 << 30, hsq=1 << 37) == INVALID      # (no overflow in the check)
