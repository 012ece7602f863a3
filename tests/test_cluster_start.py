"""A CTA's shared memory may be reached from its cluster once that CTA has started
to run.  Whether a kernel makes sure of that cannot be seen from its results, so
the order of the steps is read from the source."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "speculative_decoding_verification_04_gb300", "csrc")
# what touches a peer's shared memory
REMOTE = re.compile(r"\b(st_rank|st_rank64|ld_rank|ld_rank128|row_sync|append|list_put|list_room|command_of|merge_bins|gather_level|gather_bins|each_hit)(<[^;()]*>)?\(")


def source(name):
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def body(text, name):
    """The body of the function `name`, braces and all."""
    at = re.search(r"\b(bool|void) (__launch_bounds__\([^\n]*\) )?" + name + r"\(", text).start()
    start = text.index("{", text.index(")\n", at) if ")\n{" in text[at:at + 600] else at)
    depth = 0
    for i in range(start, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[start:i + 1]
    raise AssertionError(name)


@pytest.mark.parametrize("name", ["levels_row", "copy_row"])
def test_a_row_waits_for_its_peers_before_it_reaches_them(name):
    text = body(source("sv_filter.cuh"), name)
    assert "peers_started(C);" in text
    assert text.index("peers_started(C);") < REMOTE.search(text).start()


def test_the_filter_kernel_announces_itself_and_waits():
    text = body(source("sv_filter.cuh"), "sv_filter_kernel")
    said, waited = text.index("peers_announce(C);"), text.index("peers_started(C);")
    for path in ("levels_row<", "copy_row<"):
        assert said < text.index(path) < waited
    assert text.count("peers_announce(") == text.count("peers_started(") == 1
    # from the announcement on every way out goes through a wait: the two paths above, or the one here
    between = text[said:waited]
    assert between.count("return;") == 2 and REMOTE.search(text).start() > waited
    assert "started = true;" in between[between.index("levels_row<"):between.index("copy_row<")]
    # and none of the cluster returns before it while another one stays: the rows of a cluster are one row
    assert REMOTE.search(text[:said]) is None


@pytest.mark.parametrize("name", ["sv_pages.cuh", "sv_filter.cuh"])
def test_cluster_barriers_are_met_by_whole_warps(name):
    """barrier.cluster's .aligned form: no lane of a warp may still be on another way to it."""
    steps = [line.strip() for line in source(name).splitlines() if line.strip()]
    arrivals = ("cluster_arrive();", "cluster_arrive_relaxed();")
    at = [i for i, line in enumerate(steps) if line in arrivals]
    assert at
    for i in at:
        before = [line for line in steps[i - 4:i] if line not in ("else", "if (DRAW)", *arrivals)]
        assert before[-1] == "__syncwarp();", steps[i - 4:i + 1]
