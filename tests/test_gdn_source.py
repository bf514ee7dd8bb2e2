"""What a run cannot show of the gated delta rule's scan without a wait that gives up, read off its source (no GPU)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "recurrent_state_update_gb300", "csrc")


def function(text, name):
    """The body of the first function called name."""
    at = text.index("{", re.search(r"\b%s\([^;{]*\)\s*\{" % name, text).start())
    depth = 0
    for i in range(at, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return text[at:i + 1]


def test_the_sides_warps_agree_whether_a_wait_gave_up():
    """elect.sync needs all 32 lanes.  A wait gives up lane by lane, so what decides whether a warp reaches an
    election may hang only on waits whose outcome the lanes share."""
    text = open(os.path.join(CSRC, "gdn_scan_tc.cu")).read()
    side = function(text, "side_warps")
    assert re.search(r"if \(!bad\)", side) and "elect_one()" in side
    assert not re.search(r"\bwait_for\(", side)
    assert len(re.findall(r"\bwarp_wait_for\(", side)) >= 6
    shared = function(text, "warp_wait_for")
    assert "__all_sync(0xffffffffu, wait_for(bar, parity))" in shared


def test_both_kernels_put_their_swizzled_tiles_on_1024_byte_boundaries():
    """A swizzled operand is read right only from such a boundary; the language promises 16 bytes of the base."""
    text = open(os.path.join(CSRC, "gdn_scan_tc.cu")).read()
    for kernel, base in (("k_gdn_prep", "prep_smem"), ("k_gdn_chain", "chain_smem")):
        body = function(text, kernel)
        assert len(re.findall(r"= \*?align1024<\w+(<HEADS>)?>\(%s\)" % base, body)) == 1, kernel
        assert body.count(base) == 2  # its declaration and that
