"""Refusals of the logit rules' self-test, before any device work.  No GPU needed."""

import ctypes

from mtp_speculative_decoding_draft_gb300 import binding as bd
from mtp_speculative_decoding_draft_gb300 import build

IN, OUT = ctypes.c_void_p(1 << 20), ctypes.c_void_p(1 << 21)    # aligned, never read


def test_the_self_test_needs_a_second_row_and_a_second_array():
    build.build()
    rules, call = bd.MtpLogitRules(), bd.library().mtp_selftest_logits_wait
    assert call(1, 0, 100, rules, IN, None, OUT, None) == -1    # k = 0: no row to withhold
    assert call(1, 1, 100, rules, IN, None, IN, None) == -1     # in place: no copy to withhold
    assert call(1, 1, 100, None, IN, None, OUT, None) == -1
    assert call(0, 1, 100, rules, IN, None, OUT, None) == -1
    assert call(65, 1, 100, rules, IN, None, OUT, None) == -2    # more blocks than wait side by side
    assert call(2, 1, 100000, rules, IN, None, OUT, None) == -2
