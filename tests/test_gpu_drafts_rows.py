"""Rows of verify_tree that do not count, or hold what is not a probability (GPU)."""
import pytest
import torch

from tests.test_gpu_drafts import check_verify, drafts, run_verify

pytestmark = pytest.mark.gpu
NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("drawn", ["with", "without"])
@pytest.mark.parametrize("vocab", [300, 5000, 70001, 140000])      # by the entry's own workgroup, by launches
@pytest.mark.parametrize("bad", [NAN, INF, -INF, 1e38])
def test_draft_rows_behind_the_walk_do_not_count(drawn, vocab, bad):
    """Where no child was rejected the token comes from the target's row alone: at a leaf, and where
    the path is full, the draft's row may never have been computed."""
    for kind, counts, depth in (("chain", [5, 1, 9], 64), ("star", [4, 3, 1], 64), ("chain", [9, 7], 3), ("chain", [4], 1)):
        d = drafts(counts, vocab, kind, 5, drawn)
        d["uniform"].zero_()                             # every first child is taken
        path, lengths, token = check_verify(d, drawn, depth=depth)
        d["draft"] = d["draft"].clone()
        for i, n in enumerate(lengths):
            assert n == min(depth, counts[i] if kind == "chain" else min(2, counts[i]))
            row = d["draft"][d["cu"][i] + path[i][n - 1]]
            row[token[i]] = bad                          # where it would show, and in half of the row
            row[::2] = bad
        assert run_verify(d, drawn, depth) == (path, lengths, token)
