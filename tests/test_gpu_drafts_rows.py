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


@pytest.mark.parametrize("drawn", ["with", "without"])
@pytest.mark.parametrize("vocab", [300, 5000, 70001, 140000])
@pytest.mark.parametrize("bad", [NAN, -0.25])
def test_what_is_no_probability_in_a_draft_row_counts_as_zero(drawn, vocab, bad):
    """At a child's token and elsewhere: as if it were 0 there.  A child without a probability in either row
    is rejected and does not disturb its later siblings."""
    gone = set()
    for seed, target in ((1, 0.0), (2, 0.0), (3, None), (4, None)):
        d = drafts([6, 9, 4], vocab, "star", seed, drawn, error=2.5)
        d["uniform"] = 0.75 + d["uniform"] / 4           # most children are rejected
        clean = {**d, "draft": d["draft"].clone()}
        d["draft"] = d["draft"].clone()
        for i, a in enumerate(d["cu"][:-1]):
            x = int(d["ids"][a + 1])                     # the first child's token
            at = torch.cat((torch.arange(2, vocab, 7), torch.tensor([x])))
            at = at[~torch.isin(at, d["ids"][a + 2:d["cu"][i + 1]])]
            clean["draft"][a, at] = 0.0
            d["draft"][a, at] = bad
            if target is not None:
                d["target"][a, x] = target
        got = check_verify(clean, drawn)
        assert run_verify(d, drawn) == got
        gone |= {n for n, c in zip(got[1], (6, 9, 4)) if n < c}
    assert gone
