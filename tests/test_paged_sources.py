"""Rules of the paged kernels' sources that a run cannot show reliably: read
from the text, on the CPU."""

import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "sparse_attention_csa_gb300", "csrc")


def kernels(name):
    """{kernel: body} of a source file, comments taken out."""
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    out = {}
    for m in re.finditer(r"__global__[^;{]*?(\w+_kernel)\s*\([^{;]*\)\s*\{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        out[m.group(1)] = text[m.end():at - 1]
    return out


@pytest.mark.parametrize("name,expected", [
    ("rope.cu", {"rope_kernel", "cache_append_kernel"}),
    ("indexer_paged.cu", {"indexer_paged_score_kernel", "indexer_paged_select_kernel"}),
    ("sparse_mla_paged.cu", {"sparse_mla_paged_kernel", "sparse_mla_paged_join_kernel"}),
])
def test_nothing_is_read_before_the_wait(name, expected):
    """A kernel that may start before the one ahead of it has ended waits, on
    every path, before it touches global memory: what the wait makes visible is
    visible to the waiting grid only, not to grids that it lets start."""
    seen = kernels(name)
    assert expected <= set(seen)
    for kernel in expected:
        body = seen[kernel]
        wait = body.index("grid_dependency_wait();")
        ahead = body[:wait]
        line = ahead[ahead.rfind("\n") + 1:]
        assert line.strip() == "", f"{kernel}: the wait depends on `{line.strip()}`"
        for touch in ("__ldg", "visible_rows(", "token_keys(", "paged_seq(", "paged_row(", "report_error("):
            assert touch not in ahead, f"{kernel}: {touch} before the wait"
        assert "launch_dependents();" not in ahead, f"{kernel}: lets others start before its own wait"


def statements(body):
    return [" ".join(x.split()) for x in re.split(r"[;{}]", body) if x.strip()]


def test_waits_of_whole_warps_are_voted():
    """Where a whole warp waits in the score kernel, one lane's wait may give up
    while another's ends well. The lanes have to go on alike: a vote or a
    warp-wide load that part of a warp skips never ends. (The MMA role is one
    lane and needs no vote.)"""
    body = kernels("indexer_paged.cu")["indexer_paged_score_kernel"]
    one_lane = body[body.index("if (warp == kMmaWarp) {\n            \n"):body.index("__syncwarp();")]
    assert "if (lane == 0) {" in one_lane and "cx.wait(" in one_lane
    waits = [x for x in statements(body.replace(one_lane, "")) if "cx.wait(" in x]
    assert len(waits) == 4
    for x in waits:
        assert "__all_sync(0xffffffffu, cx.wait(" in x, x


def test_selection_ranks_nan_like_it_counts_it():
    """The selection writes the rows whose key lies above the border's and
    counts them by linear bins: a NaN has one place in both (its own key, no
    bins). float_key alone ranks it below zero."""
    body = kernels("indexer_paged.cu")["indexer_paged_select_kernel"]
    assert "row_key(" in body and "float_key(" not in body
