"""step_tree for every type, rule, key width, range of value widths and bound on a tree's nodes: the
kernel has an instance for each (GPU)."""
import pytest
import torch

from tests.test_gpu_drafts import RULES, TYPES, check_tree, run_tree

pytestmark = pytest.mark.gpu
# up to 16, 32, 48 and 64 nodes take bodies of their own
COUNTS = {16: [16, 5, 1], 32: [32, 17, 9], 64: [64, 33, 48, 20, 3, 50]}


@pytest.mark.parametrize("bound", COUNTS)
@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
@pytest.mark.parametrize("shape", [(2, 1, 64, 64), (2, 2, 64, 33), (2, 1, 64, 136), (2, 1, 128, 64), (4, 2, 128, 24),
                                   (2, 2, 128, 130)], ids=lambda s: "x".join(map(str, s)))
def test_every_instance(bound, io, delta, diag, shape):
    counts = COUNTS[bound]
    slots = [(3 * i + 1) % 7 for i in range(len(counts))]
    for kind, seed in (("random", 3), ("chain", 4)):
        def edit(x):                                     # no, a negative and a full decay; nothing written; fast decays
            if kind == "random":
                x["alpha"][2], x["alpha"][counts[0] + 3], x["alpha"][-2] = 0.0, -0.5, 1.0
                x["beta"][1] = 0.0
            else:
                x["alpha"][::5] = x["alpha"][::5] ** 40
        o, want, mag, T = run_tree(counts, kind, *shape, TYPES[io], delta, diag, slots=slots, n_slots=8,
                                   fresh=[i == 1 for i in range(len(counts))], max_nodes=bound, seed=seed, edit=edit)
        check_tree(o, want, mag, T, shape[2], TYPES[io], delta)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
@pytest.mark.parametrize("shape", [(2, 1, 64, 136), (4, 2, 128, 64)], ids=lambda s: "x".join(map(str, s)))
def test_strides_at_four_tiles(io, delta, diag, shape):
    o, want, mag, T = run_tree([40, 9, 64], "random", *shape, TYPES[io], delta, diag, pad=8, o_pad=3)
    check_tree(o, want, mag, T, shape[2], TYPES[io], delta)
