"""What the merge of new tokens' partial results reads: a cut for each stream and class, in every case of the call's own.

The merge runs behind the attention kernel whatever became of it, and takes the bounds of its loops and its
addresses from the cuts in the workspace, which may hold anything before a call. A schedule that gives up in a
bounded wait must therefore have written all of its cuts before. That needs an expired wait to happen on a GPU, so
it is read from the source here.
"""
import os
import re

import medusa_speculative_decoding_heads_gb300 as package

CSRC = os.path.join(os.path.dirname(package.__file__), "csrc")


def schedule():
    """The source of the schedule of new tokens, without comments."""
    with open(os.path.join(CSRC, "rows_tc.cu"), encoding="utf-8") as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    return text[text.index("if (kChunk && warp >= kPlanWarp) {"):text.index("} else if (warp == kPlanWarp) {")]


def test_cuts_of_both_classes_are_written_ahead_of_every_wait():
    text = schedule()
    # the first thing that may leave the schedule is the class loop, which ends with `ok`
    ahead = text[:text.index("for (int single")]
    calls = ahead.replace(ahead[ahead.index("auto free_slot"):ahead.index("};", ahead.index("auto free_slot"))], "")
    assert "mbar_wait" not in calls and "free_slot()" not in calls
    resets = re.findall(r"(?:if \(([^;{]*)\)\s*)?a\.cuts\[([^\]]*)\] = ChunkCut\{0, 0, 0, 0\};", ahead)
    where = {index.replace(" ", ""): guard for guard, index in resets}
    assert set(where) == {"blockIdx.x", "sp.pair_streams+blockIdx.x"}
    assert "sp.pair_streams" in where["blockIdx.x"]   # (without pairs that place is a single tile's)
    assert "pair_streams" not in where["sp.pair_streams+blockIdx.x"]
    # and none is put back to nothing behind a wait
    assert "ChunkCut{0, 0, 0, 0}" not in text[len(ahead):]
