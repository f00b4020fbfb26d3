"""What is not finite, or leaves fp32's range on the way, in step_tree: it reaches its node and those
behind it, and nothing else (GPU)."""
import pytest
import torch

from tests.drafts_ref import trees
from tests.test_gpu_drafts import DEV, RULES, TYPES, check_tree, run_tree

pytestmark = pytest.mark.gpu


def family(n, seed, nodes):
    """Parents of a random tree in which each of nodes continues the one before it, and the nodes
    from each of them on."""
    parents = trees([n], "random", seed)
    for a, b in zip(nodes, nodes[1:]):
        parents[b] = a
    behind = []
    for x in nodes:
        one = {x}
        for j in range(n):
            if parents[j] in one:
                one.add(j)
        behind.append(one)
    return parents, behind


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
@pytest.mark.parametrize("n,nodes", [(14, (4, 5)), (40, (4, 5)), (40, (4, 20)), (40, (18, 21)), (64, (33, 40)), (64, (20, 50))])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_a_write_that_overflows_stays_on_its_paths(io, delta, diag, n, nodes, dk, dv):
    """Under the delta rule two large gates, one behind the other, whose writes' product leaves fp32's
    range though neither of them does; a gate whose write is finite in fp32 and not as bf16."""
    parents, behind = family(n, 5, nodes)
    args = ("random", 2, 2, dk, dv, TYPES[io], delta, diag)
    for gates in ([2.0 ** 70, 2.0 ** 70], [0.5, float.fromhex("0x1.ff8p127")]):
        def edit(x):
            for node, gate in zip(nodes, gates):
                x["beta"][node, 0] = gate
                x["v"][node, 0] = 1
        o, _, _, _ = run_tree([n], *args, edit=edit, parents=parents)
        clean, ref, mag, T = run_tree([n], *args, parents=parents)
        keep = torch.ones_like(ref, dtype=torch.bool)
        keep[sorted(behind[0]), 0] = False
        assert len(behind[0]) < n - 3
        check_tree(torch.where(keep.to(DEV), o, float("nan")), torch.where(keep, ref, float("nan")), mag, T, dk, TYPES[io], delta)
        if delta and gates[0] > 1:                       # w of the second node is beyond fp32
            assert not bool(o[sorted(behind[1]), 0].isfinite().any())


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("n,nodes", [(16, (4, 9)), (32, (4, 18)), (40, (20, 37)), (64, (37, 60)), (64, (3, 50))])
@pytest.mark.parametrize("dk,dv", [(64, 64), (128, 128)])
def test_every_node_behind_one_that_is_not_finite_is_not(io, delta, diag, bad, n, nodes, dk, dv):
    """On its own tile and on later ones; the other nodes stay as they are."""
    parents, behind = family(n, 7, nodes)
    spoilt, behind = nodes[0], sorted(behind[0])
    args = ("random", 2, 2, dk, dv, TYPES[io], delta, diag)
    clean, ref, mag, T = run_tree([n], *args, parents=parents)
    for name in ("q", "k", "v", "alpha", "beta"):
        def edit(x):
            if name == "v":
                x["v"][spoilt, 0, 3] = bad
            elif name in ("q", "k"):
                x[name][spoilt, 0, 5] = bad
            else:
                x[name][spoilt, 0] = bad
        o, _, _, _ = run_tree([n], *args, edit=edit, parents=parents)
        rows = [spoilt] if name == "q" else behind
        gone = torch.zeros_like(ref, dtype=torch.bool)
        for j in rows:
            gone[j, 0, 3 if name == "v" else slice(None)] = True
        assert not bool(o.cpu()[gone].isfinite().any()), name
        check_tree(torch.where(gone.to(DEV), float("nan"), o), torch.where(gone, float("nan"), ref), mag, T, dk, TYPES[io], delta)
