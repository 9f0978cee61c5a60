"""The pairs' kernels, read as text: what crosses from one CTA to the other.  No GPU needed."""

import pathlib
import re

import pytest

CSRC = pathlib.Path(__file__).parent.parent / "mtp_speculative_decoding_draft_gb300" / "csrc"


@pytest.mark.parametrize("name,bars", [("latent_attn_pair.cu", {"p_full", "o_empty", "v_full"}), ("latent_heads.cu", {"tfree"})])
def test_arrivals_from_the_other_cta_are_waited_for_at_cluster_scope(name, bars):
    """A wait at CTA scope does not synchronise with a thread of another CTA: the softmax weights and
    sums (p_full), accumulators given back (o_empty, tfree) and cleared values (v_full) could be
    used before they are there."""
    text = (CSRC / name).read_text()
    far = set(re.findall(r"mbar_arrive_cluster_relaxed\(\s*dsmem_addr\(&?(\w+)", text))
    far |= set(re.findall(r"mbar_arrive_remote\(&?(\w+)", text))
    assert far == bars
    for bar in far:
        assert re.search(r"(await|mbar_wait_cluster)\(&?%s\b" % bar, text), bar
    for helper in re.findall(r"auto await = [^;]*;", text):
        assert "mbar_wait_cluster(bar, parity" in helper
    # What is left at CTA scope: values that a CTA brings and clears for itself, and, in the products, the
    # wait for the last of them, behind which nothing is read.
    assert set(re.findall(r"\bmbar_wait\(&?(\w+)", text)) <= {"zbar"}
    assert set(re.findall(r"mbar_sleep_wait\(&?(\w+)", text)) <= {"drain"}


def test_tensor_memory_is_handed_over_between_fences():
    """Stores complete, the fence, the warp together, the arrival; the wait, the fence, the product."""
    text = (CSRC / "latent_attn_pair.cu").read_text()
    assert re.search(r"tmem_wait_st\(\);\s*tc_fence_before\(\);\s*__syncwarp\(\);(\s*//[^\n]*)*\s*if \(lane == 0\) "
                     r"mbar_arrive_cluster_relaxed\(dsmem_addr\(&p_full", text)
    assert re.search(r"await\(&p_full[^;]*;\s*await\(&v_full[^;]*;\s*tc_fence_after\(\);", text)
