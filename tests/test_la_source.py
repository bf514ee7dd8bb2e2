"""What a run cannot show of linear attention's scan without a wait that gives up, read off its source (no GPU)."""
import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "recurrent_state_update_gb300", "csrc")


def source():
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "la_scan_tc.cu")).read())


def test_every_wait_has_one_outcome_for_its_warp():
    """elect.sync and the tensor-memory instructions need all 32 lanes, so whether a warp reaches them may hang only on
    outcomes that its lanes share."""
    text = source()
    assert "ok = __all_sync(0xffffffffu, ok);" in text
    assert not re.search(r"\bmbar_wait\(", text)
    polls = [m.start() for m in re.finditer(r"mbar_try_wait\(", text)]
    assert len(polls) == 2  # the warp's wait, and what drains after a failure


def test_the_outputs_warps_leave_together():
    """They meet at a barrier of their own: a warp that left alone would keep the others there."""
    text = source()
    a = text.index("outputs_sync_or(!wait(B_Y2, g))")
    b = text.index("more_registers<kStateRegs>();")
    body = text[a:b]
    assert not re.search(r"(?<!outputs_sync_or\(!)wait\(B_", body)
    assert len(re.findall(r"outputs_sync_or\(!wait\(", body)) == 2


def test_register_shares_stay_within_the_launch():
    """setmaxnreg.inc waits for ever for what the launch did not give the block."""
    text = source()
    value = {n: int(v) for n, v in re.findall(r"\b(k\w*Regs) = (\d+)", text)}
    assert value["kScoreRegs"] + value["kOutRegs"] + value["kStateRegs"] + value["kKeyRegs"] + value["kIssueRegs"] <= 5 * value["kRegs"]
    assert value["kSumRegs"] + 2 * value["kScaleRegs"] + value["kSegIssueRegs"] <= 4 * value["kSegRegs"]
    assert all(v % 8 == 0 for v in value.values())
    for regs in ("kRegs", "kSegRegs"):  # what the compiler made of it is checked before each launch
        assert re.search(r"ready\(reinterpret_cast<const void \*>\(kern\), smem, %s\)" % regs, text)


def test_the_ring_of_units_counts_its_phases():
    """Slot and phase of a turn, as the warp that gives out and those that take compute them; a fresh mbarrier passes a wait
    for parity 1, so that a phase counted wrong reads a slot before it is written."""
    text = source()
    assert "const int at_ring = k % kRing, use = k / kRing;" in text and "const int k = units.k % kRing;" in text
    ring = int(re.search(r"constexpr int kRing = (\d+);", text).group(1))
    completed = [0] * ring
    for k in range(5 * ring):
        slot, use = k % ring, k // ring
        assert (completed[slot] - 1) & 1 != use & 1  # not yet given out: the wait holds
        completed[slot] += 1
        assert (completed[slot] - 1) & 1 == use & 1  # given out: it passes


def braces(text, at):
    """The text within the braces that open first from `at` on, and where they end."""
    a = text.index("{", at)
    depth = 0
    for i in range(a, len(text)):
        depth += (text[i] == "{") - (text[i] == "}")
        if depth == 0:
            return text[a + 1:i], i + 1


def test_a_warpgroup_changes_its_registers_in_one_instruction():
    """All warps of a warpgroup have to execute the same setmaxnreg, before anything they do not do together; what a group of
    four asks for is free only once every group has given up its share."""
    text = source()
    sites = r"\b(?:fewer|more)_registers<\w+>\(\);"
    for kernel, groups in (("k_la_chain", 5), ("k_la_segment", 4)):
        body, _ = braces(text, re.search(r"\b%s\(const ScanParams p" % kernel, text).end())
        at, warps, shared = re.search(r"\n    if \(warp < \d+\) \{", body).start(), 0, 0
        while True:
            head = re.match(r"\s*(?:else )?(?:if \(warp < (\d+)\) |(?=\{))", body[at:])
            assert head, (kernel, "a warpgroup's warps go different ways", body[at:at + 40])
            branch, end = braces(body, at)
            upto = int(head.group(1)) if head.group(1) else 4 * groups
            assert upto % 4 == 0 and warps < upto  # whole warpgroups
            assert len(re.findall(sites, branch)) == 1 and re.match(r"\s*" + sites, branch), (kernel, warps)
            warps, shared = upto, shared + 1
            tail = re.match(r"\s*else ", body[end:])
            if not tail:
                break
            at = end
        assert warps == 4 * groups and len(re.findall(sites, body)) == shared
