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


def test_pages_are_refused_to_a_module_per_depth(module, monkeypatch):
    """The paged chain would run the first module at every depth."""
    def fail(*a, **k):
        raise AssertionError("reached the library")
    for name in ("make_paged_cache", "paged_workspace_size", "mtp_draft_paged", "spec_step_paged"):
        monkeypatch.setattr(bd, name, fail)
    module.extra = [{"E": None}]
    with pytest.raises(ValueError, match="one module"):
        module.set_pages(None, None, None)
    assert module.ws_paged is None
    for call in (lambda: module.draft_paged(1.0, 0), lambda: module.step_paged(1.0, 0, None)):
        with pytest.raises(ValueError, match="set_pages"):
            call()


def test_new_pages_keep_the_workspace(module, monkeypatch):
    """A program that grows its page table calls set_pages again and again."""
    class Guard:
        made = 0

        def alloc(self, name, numel, dtype):
            self.made += 1
            return (name, numel)
    monkeypatch.setattr(bd, "make_paged_cache", lambda *pools: pools)
    monkeypatch.setattr(bd, "paged_workspace_size", lambda dims, k: 1024)
    module.dims, module.k, module.guard = None, 3, Guard()
    for table in ("small", "larger"):
        module.set_pages("k", "v", table, window=7, sinks=1)
        assert module.cache == ("k", "v", table) and module.ws_paged == ("paged workspace", 1024)
    assert module.guard.made == 1
