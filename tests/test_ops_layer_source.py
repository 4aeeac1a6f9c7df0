"""What the attention kernels' source has to hold for their hand-overs between threads, where a
mistake would show only by chance on a GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "gated_delta_rule_varlen_gb300", "csrc")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


# Barriers by which tensor memory changes hands, between the threads that issue products and those
# that read and write it (not those of the rings of tiles in shared memory).
HANDOVER = {"gdr_attn_fwd.cu": "s_full|p_full|o_full|o_empty",
            "gdr_attn_bwd.cu": "s_full|p_full|dp_full|dp_read|ds_full|dq_done|acc_full|acc_empty"}
USES = re.compile(r"tc_fence_after\(\)|\bmma_(?:ss|ts|rows|sum)\b|\bscore\(|\bgrad\(\)|\bload_cols\(|\btmem_ld\d+\(|\bstore16\(")


@pytest.mark.parametrize("name", sorted(HANDOVER))
def test_tensor_memory_is_used_after_a_fence(name):
    # tcgen05 operations of different threads are ordered by a barrier and the fence behind its wait
    text, found = source(name), []
    for m in re.finditer(r"warp_wait(?:_all)?\([^;]*&s\.(%s)\b[^;]*;" % HANDOVER[name], text):
        use = USES.search(text, m.end())
        found.append(m.group(1))
        assert use and use.group(0).startswith("tc_fence_after"), (m.group(0), use and use.group(0))
    assert len(found) >= 4


def test_dkv_begins_early_only_behind_dq():
    # k_attn_dkv reads the documents' bounds and starts its loads before it waits for the kernel before:
    # only where that is k_attn_dq (or follows it), all of whose threads wait for what came before first
    text = source("gdr_attn_bwd.cu")
    launches = re.findall(r"go\(k_attn_dkv<[^>]*>, b\d, blocks, f, st(?:, (\w+))?\)", text)
    assert len(launches) == 4 and set(launches) == {"early"}
    assert re.search(r"const bool early = qblocks > 0;", text)
    dq = text[text.index("k_attn_dq(const"):text.index("k_attn_dkv(const")]
    assert dq.index("previous_ended();") < min(dq.index("next_may_start();"), dq.index("BlockFinder"), dq.index("if (warp >= WORKERS)"))


def test_blocks_are_found_in_any_order():
    # clusterlaunchcontrol.try_cancel answers with any block that has not begun; a search that only
    # went on would compute a place before its documents
    text = source("gdr_attn.cuh")
    find = text[text.index("AttnBlock find(int want)"):]
    assert re.match(r"AttnBlock find\(int want\) \{\s*if \(want < before\) \{\s*before = 0;\s*load\(0\);\s*\}", find)


def test_the_scan_waits_by_tries():
    # the clock's instructions in its loops cost the scan 5% (32768 tokens 441 -> 466 us)
    text = source("gdr_ssm_tc.cu")
    waits = re.findall(r"\b(?:warp_wait(?:_all)?|wait_or_abort|try_phase)\b(<\w+>)?\(", text)
    assert len(waits) > 20 and set(waits) == {"<ByTries>"}


def test_the_wait_for_an_items_end_grows_with_the_item():
    # an item's steps are waited for each within the limit; the warp that asks for items waits for all
    # of them together, of which a document of some 10^7 tokens has more than fit in it
    text = source("gdr_attn_tc.cuh")
    run = text[text.index("void run("):text.index("bool take(")]
    assert "kWaitNs * (1 + (uint64_t)w.steps())" in run and re.search(r"warp_wait_within\(limit, abort, Phase\{&wanted,", run)
    assert len(re.findall(r"int steps\(\) const", source("gdr_attn_fwd.cu") + source("gdr_attn_bwd.cu"))) == 3
