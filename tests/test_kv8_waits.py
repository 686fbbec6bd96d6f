"""Waits that may give up and steps that all threads of a warp or block take together, in the sources of the 8-bit
cache's kernels, without a GPU.

Every thread's wait (mbar_wait_bounded) has its own clock.  Where a warp-wide or block-wide step follows, the threads
either agree on the answer first, by a vote of the warp, or all go on."""

import os
import re

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "tree_speculative_decoding_split_gb300",
                    "csrc")


def _code(name):
    return re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())


def test_append_threads_stay_for_their_blocks_steps():
    """No thread leaves the rounds; behind a wait that gave up nothing is asked for or written."""
    code = _code("kv8_append.cu")
    loop = code[code.index("for (int base = i0, turn = 0;"): code.index("struct AppendShape")]
    assert not re.search(r"\breturn;", loop) and not re.search(r"\bbreak;", loop)
    assert "if (!mbar_wait_bounded(&s_full[stage], phase, &s_gave_up)) s_gave_up = 1;" in loop
    barrier, skip = loop.index("__syncthreads()"), loop.index("if (item >= i1 || (TMA && s_gave_up)) continue;")
    assert loop.index("__reduce_max_sync") < barrier < skip < loop.index("store_codes")
    assert "base + kStages * groups < i1 && !s_gave_up) fetch(" in loop


def test_few_rows_boxes_end_for_the_whole_warp():
    code = _code("attention_kv8.cu")
    loop = code[code.index("for (; i < mine; ++i) {"):]
    loop = loop[: loop.index("softmax_step<RN, NT>(y, st, o, inv_vs")]
    wait = loop.index("mbar_wait_bounded")
    assert re.search(r"if \(!__all_sync\(0xffffffffu, mbar_wait_bounded\(&s_full\[warp\]\[s\], \(i / kStagesR\) & 1, &s_abort\)\)\) "
                     r"\{\s*ok = false;\s*break;", loop)
    assert loop.count("break;") == 1 and loop.index("break;") > wait
    assert "for (int j = i; j < min(mine, i + kStagesR); ++j)" in code
