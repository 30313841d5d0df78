"""The bounded waits of whole warps in the tensor-core kernels: one answer for all lanes.

Each lane polls the barrier and the abort flag for itself, so while a wait
expires one lane may see the barrier complete and another the flag.  A lane that
gives up goes to the CTA's last barrier; lanes that went on would stop at the next
warp-wide instruction and wait there for it without limit.  So every wait of a whole warp has to
end in a vote, which is checked in the source: no run can be made to show it
without a GPU that hangs."""
import os
import re

import pytest

from trie_constrained_beam_fr_b200 import build

WAIT = re.compile(r"\b(tc_wait|gm_wait_pair)\(")


def _source(name):
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _after(text, start, end):
    i = text.index(start)
    return text[i:text.index(end, i)]


@pytest.mark.parametrize("name,end", [("fr_gemm.cuh", "tc_fence_before"), ("fr_lmhead.cu", "__syncthreads")])
def test_the_epilogue_warps_waits_vote(name, end):
    part = _after(_source(name), "warp >= 4", end)
    waits = list(WAIT.finditer(part))
    votes = re.findall(r"\btc_wait_warp\(", part)
    assert not waits and len(votes) == 1


def test_the_vote_is_over_the_whole_warp():
    body = _after(_source("fr_tc.cuh"), "bool tc_wait_warp(", "\n}")
    assert re.search(r"return __all_sync\(0xffffffffu, tc_wait\(", body)


def test_a_published_tile_is_waited_for_together():
    """Of `next`: its answer is put to the vote where whole warps call it."""
    part = _after(_source("fr_gemm.cuh"), "const auto next =", "};")
    answer = re.search(r"(?:const )?bool (\w+) = rank == 0 \? tc_wait\(", part)
    assert answer, "the wait's answer has a name"
    assert re.search(r"whole \? __all_sync\(0xffffffffu, %s\) : %s" % (answer.group(1), answer.group(1)), part)
    assert len(WAIT.findall(part)) == 2
