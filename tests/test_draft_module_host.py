"""DraftModule's bookkeeping around the paged calls, with the library's calls replaced
by fakes.  No GPU needed."""

import pytest

from mtp_speculative_decoding_draft_gb300 import binding as bd
from mtp_speculative_decoding_draft_gb300.model import DraftModule


@pytest.fixture
def module():
    m = DraftModule.__new__(DraftModule)
    m.ws, m.ws_paged, m.mods, m.extra = "contiguous", None, None, []
    return m


@pytest.mark.parametrize("bits", [{}, {"paged": bd.STATUS_BAD_CTX}, {"contiguous": bd.STATUS_BAD_TOKEN},
                                  {"contiguous": bd.STATUS_BAD_TOKEN, "paged": bd.STATUS_BAD_PAGE | bd.STATUS_TIMEOUT}])
def test_status_covers_both_workspaces(module, monkeypatch, bits):
    monkeypatch.setattr(bd, "get_status", lambda ws, stream=None: bits.get(ws, 0))
    assert module.status() == bits.get("contiguous", 0)          # no pages yet
    module.ws_paged = "paged"
    assert module.status() == bits.get("contiguous", 0) | bits.get("paged", 0)
