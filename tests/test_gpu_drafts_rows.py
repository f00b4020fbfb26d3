"""Rows of verify_tree that do not count, or hold what is not a probability (GPU)."""
import pytest
import torch

import quantized_recurrent_state_amd as lsq
from tests.test_gpu_drafts import DEV, check_verify, drafts, i32, run_verify

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


def rest_ref(d, depth):
    """verify_tree of siblings drawn without replacement, in 64 bits, with Q the draft's mass that is not tried
    yet wherever 1 - q(x_1) - ... is below 1/16."""
    paths, lengths, tokens = [], [], []
    for i, a in enumerate(d["cu"][:-1]):
        n, path = d["cu"][i + 1] - a, [0]
        while True:
            row, tried, c, T, Q, taken = a + path[-1], [], 0.0, 1.0, 1.0, None
            p, q = d["target"][row].double(), d["draft"][row].double()
            for j in range(path[-1] + 1, n) if len(path) < depth else ():
                if d["parents"][a + j] != path[-1]:
                    continue
                x = int(d["ids"][a + j])
                if float(d["uniform"][a + j]) * T * float(q[x]) < max(float(p[x]) - c * float(q[x]), 0.0) * Q:
                    taken = j
                    break
                tried.append(x)
                c += T / Q
                T = float((p - c * q).clamp(min=0).sum())
                Q = Q - float(q[x])
                if Q < 1.0 / 16:
                    left = q.clone()
                    left[tried] = 0.0
                    Q = float(left.sum())
            if taken is None:
                break
            path.append(taken)
        cum = (p - c * q).clamp(min=0).cumsum(0)
        tokens.append(int((cum <= float(d["uniform_next"][i]) * float(cum[-1])).sum()))
        paths.append(path + [-1] * (depth - len(path)))
        lengths.append(len(path))
    return paths, lengths, tokens


def nearly_certain(d, little, scale=1.0):
    """Draft rows that leave `little` to all tokens but the first child's, which the target never has."""
    rest = d["draft"].double()
    first = torch.zeros(len(rest), dtype=torch.long)
    used = set()
    for a, b in zip(d["cu"], d["cu"][1:]):
        for j in range(a + 1, b):
            row = a + d["parents"][j]
            if row not in used:
                used.add(row)
                first[row] = int(d["ids"][j])
    at = torch.arange(len(rest))
    rest[at, first] = 0.0
    rest *= little / rest.sum(-1, keepdim=True)
    rest[at, first] = 1.0 - little
    d["draft"] = (rest * scale).float()
    d["target"][at, first] = 0.0
    d["target"] = (d["target"].double() / d["target"].double().sum(-1, keepdim=True)).float()
    d["uniform"] = 0.9 + d["uniform"] / 10


@pytest.mark.parametrize("vocab", [4099, 32000, 70001, 131073])
@pytest.mark.parametrize("counts", [[3] * 12, [6] * 8, [9, 12, 3, 17]], ids=str)
@pytest.mark.parametrize("little", [0.05, 7e-4, 2e-6, 2e-7])
@pytest.mark.parametrize("scale", [1.0, 1.0 + 3e-5, 1.0 - 3e-5])
def test_little_left_of_a_draft_without_replacement(vocab, counts, little, scale):
    """A draft that is nearly certain of its first token, which fails; its later siblings are drawn from the
    little that is left, of rows that sum to one but for `scale` and their rounding."""
    for seed in (1, 2):
        d = drafts(counts, vocab, "star" if seed == 1 else "random", seed, "without", error=2.0)
        for a, c in zip(d["cu"], counts):
            d["parents"][a] = -1
            d["parents"][a + 1:a + c] = [max(0, p) for p in d["parents"][a + 1:a + c]]
        nearly_certain(d, little, scale)
        got = run_verify(d, "without", 5)
        assert got == rest_ref(d, 5)


@pytest.mark.parametrize("vocab", [32000, 70001])
def test_a_replayed_graph_with_and_without_little_left(vocab):
    counts = [9, 12, 3, 17]

    def batch(seed, little):
        d = drafts(counts, vocab, "star", seed, "without", error=2.0)
        if little:
            nearly_certain(d, little)
        return d

    d = batch(1, 0)
    names = ("target", "draft", "ids", "uniform", "uniform_next")
    rows = {n: d[n].to(DEV) for n in names}
    tree, cu = i32(*d["parents"]), i32(*d["cu"])

    def run():
        return lsq.verify_tree(rows["target"], rows["ids"], tree, cu, rows["uniform"], rows["uniform_next"],
                               draft=rows["draft"], replacement=False, depth=5)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    torch.cuda.current_stream().wait_stream(stream)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run()
    for seed, little in ((2, 2e-6), (3, 0), (4, 7e-4), (5, 0), (6, 0.05)):
        d = batch(seed, little)
        for n in names:
            rows[n].copy_(d[n])
        g.replay()
        torch.cuda.synchronize()
        got = tuple(t.tolist() for t in out)
        assert got == rest_ref(d, 5)
        assert got == tuple(t.tolist() for t in run())
