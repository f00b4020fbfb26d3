"""Drafted tokens on the GPU: step_tree, accept_path and verify_tree.

Tolerances (fixed before the first run).  u = 2^-24.  With every term of the recurrence taken by its
absolute value (the references' second result, A) a path of T nodes in fp32 is off by at most
(3 T + dk + 16) u A: per node a decay, a gate and a write, dk terms of a dot product, and a few
for their joining; the output is then rounded once, half a step of its type.  The outputs of 16-bit
types may be formed from operands held to 16 bits: 2^-16 A (bf16) or 3 2^-16 A (binary16, whose q is
two parts as well) beside.  The delta rule counts both terms of v - S k in A; as A then grows with the
depth, its outputs and states are also held in the 2-norm, where many independent roundings stay far
below their worst case: 64 u, and the operands' bound, beside the half step.
A 16-bit output's half step is taken at the largest value it may have been rounded from.
"""
import pytest
import torch

import quantized_recurrent_state_amd as lsq
from tests.drafts_ref import path_ref, tree_ref, trees, verify_ref
from tests.slots_ref import U32, half_step, rel, tokens
from tests.test_gpu_slots import SHAPES, offsets, state

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
OPERANDS = {torch.bfloat16: 2.0 ** -16, torch.float16: 3 * 2.0 ** -16, torch.float32: 0.0}
RULES = [(0, 0), (1, 0), (0, 1), (1, 1)]


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def check_tree(o, want, mag, T, dk, dtype, delta):
    o = o.double().cpu()
    live = ~want.isnan()
    assert bool(o[live].isfinite().all())
    lost = (OPERANDS[dtype] + (3 * T + dk + 16) * U32) * mag
    bound = lost + half_step(dtype) * (want.abs() + lost)
    if dtype == torch.float16:
        bound = bound + 2.0 ** -25           # half a step of a subnormal
    over = ((o - want).abs() - bound)[live]
    assert over.numel() == 0 or float(over.max()) <= 0, f"off by {float(over.max())} over the bound"
    if live.any():
        assert rel(o[live], want[live]) <= half_step(dtype) + OPERANDS[dtype] + (64 if delta else 16) * U32


def run_tree(counts, shape, heads, qk_heads, dk, dv, dtype, delta=0, diag=0, slots=None, fresh=None,
             n_slots=None, pad=0, o_pad=0, tail=0, seed=3, max_nodes=64, edit=None, parents=None):
    cu = offsets(counts)
    n = cu[-1] + tail
    slots = list(range(len(counts))) if slots is None else slots
    st, S = state(n_slots or max(slots + [0]) + 2, heads, dk, dv, delta, diag)
    x = dict(zip(("q", "k", "v", "alpha", "beta"), tokens(n, heads, qk_heads, dk, dv, dtype, seed, diag, False, pad)))
    parents = trees(counts, shape, seed) if parents is None else parents
    if edit:
        edit(x)

    def dev(t):
        if pad and t.dim() == 3 and t.dtype == dtype and t.shape[0]:
            base = t.as_strided((t.shape[0], t.stride(0)), (t.stride(0), 1))
            return base.to(DEV)[:, :t.shape[1] * t.shape[2]].unflatten(1, t.shape[1:])
        return t.to(DEV)

    wide = torch.full((n, heads * dv + o_pad), float("nan"), dtype=dtype, device=DEV)
    o = wide[:, :heads * dv].unflatten(1, (heads, dv))
    before = st.f32.clone()
    got = st.step_tree(*(dev(t) for t in x.values()), i32(*cu), i32(*(parents + [7] * tail)), slots=i32(*slots),
                       fresh=None if fresh is None else torch.tensor(fresh, device=DEV), max_nodes=max_nodes, o=o)
    assert got is o
    assert torch.equal(st.f32, before), "the state was written"
    want, mag = tree_ref(S, slots, fresh, cu, parents, *x.values(), delta=delta)
    if o_pad:
        assert bool(wide[:, heads * dv:].isnan().all())
    return o, want, mag, max(counts)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_tree_shapes(io, delta, diag, shape):
    o, want, mag, T = run_tree([7, 1, 20], "random", *shape, TYPES[io], delta, diag, slots=[2, 0, 3],
                               fresh=[False, True, False], max_nodes=20)
    check_tree(o, want, mag, T, shape[2], TYPES[io], delta)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("n", [1, 2, 3, 8, 15, 16, 17, 31, 32, 33, 47, 48, 49, 63, 64])
def test_tree_sizes(io, n):
    for kind, delta, diag in (("chain", 1, 0), ("random", 0, 0), ("star", 1, 1), ("forest", 0, 1), ("random", 1, 0)):
        o, want, mag, T = run_tree([n], kind, 2, 1, 64, 64, TYPES[io], delta, diag, max_nodes=n)
        check_tree(o, want, mag, T, 64, TYPES[io], delta)
    o, want, mag, T = run_tree([n], "chain", 1, 1, 128, 128, TYPES[io], 1, n % 2, fresh=[True])
    check_tree(o, want, mag, T, 128, TYPES[io], 1)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
def test_tree_empty_padded_and_outside(io, delta, diag):
    # empty trees, a padded entry, rows behind the last tree, one slot read by two entries
    o, want, mag, T = run_tree([0, 9, 0, 17, 5, 33], "random", 2, 2, 64, 64, TYPES[io], delta, diag,
                               slots=[4, 1, 0, -1, 6, 1], fresh=[True, False, False, True, False, False], tail=9)
    check_tree(o, want, mag, T, 64, TYPES[io], delta)
    assert bool(o.cpu()[want.isnan()].isnan().all()), "a row that no tree owns was written"


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
def test_tree_strided_rows(io, delta, diag):
    # q, k, v as slices of a wider projection, o inside a wider row
    for counts, shape in (([12, 20], (2, 2, 64, 64)), ([40, 9], (2, 1, 128, 72)), ([5], (1, 1, 64, 33))):
        o, want, mag, T = run_tree(counts, "random", *shape, TYPES[io], delta, diag, pad=8, o_pad=3)
        check_tree(o, want, mag, T, shape[2], TYPES[io], delta)


def test_tree_many_entries():
    counts = [(7 * i) % 23 for i in range(150)]
    o, want, mag, T = run_tree(counts, "random", 1, 1, 64, 64, torch.bfloat16, 1, 0,
                               slots=[(11 * i) % 160 for i in range(150)], n_slots=160, max_nodes=22)
    check_tree(o, want, mag, T, 64, torch.bfloat16, 1)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
def test_tree_resets_and_signs(io, delta, diag):
    # alpha 0 forgets what was before, a negative one is taken as it stands, beta 0 writes nothing
    def edit(x):
        x["alpha"][3] = 0.0
        x["alpha"][7] = -0.5
        x["beta"][5] = 0.0
        x["alpha"][20] = 1.0
    for kind in ("chain", "random"):
        o, want, mag, T = run_tree([24], kind, 2, 1, 64, 64, TYPES[io], delta, diag, edit=edit)
        check_tree(o, want, mag, T, 64, TYPES[io], delta)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("n", [14, 40])
def test_tree_what_is_not_finite_stays_on_its_paths(io, delta, diag, bad, n):
    """A node's input that is not finite reaches the nodes behind it alone: every other row is what
    it is without it, and its own is not finite."""
    spoilt = 4
    parents = trees([n], "random", 5)
    parents[spoilt + 1] = spoilt
    behind = {spoilt}
    for j in range(n):
        if parents[j] in behind:
            behind.add(j)
    others = [j for j in range(n) if j not in behind]
    assert others[-1] > spoilt
    for name in ("q", "k", "v", "alpha", "beta"):
        def edit(x):
            if name == "v":
                x["v"][spoilt, 0, 3] = bad                # one value column of one head
            elif name in ("q", "k"):
                x[name][spoilt, 0, 5] = bad
            else:
                x[name][spoilt, 0] = bad
        args = (("random"), 2, 2, 64, 64, TYPES[io], delta, diag)
        o, want, mag, T = run_tree([n], *args, edit=edit, parents=parents)
        clean, ref, mag, T = run_tree([n], *args, parents=parents)
        keep = torch.zeros_like(ref, dtype=torch.bool)
        keep[others] = True
        keep[:, 1] = True                                # the other head
        if name == "v":
            keep[:, 0, :3] = keep[:, 0, 4:] = True       # the other columns
        if name == "q":
            keep[[j for j in range(n) if j != spoilt]] = True
        only = torch.where(keep, ref, float("nan"))
        check_tree(torch.where(keep.to(DEV), o, float("nan")), only, mag, T, 64, TYPES[io], delta)
        assert not bool(o[spoilt, 0, 3].isfinite())


def test_tree_fresh_ignores_a_spoilt_slot():
    st, S = state(3, 2, 64, 64, 1)
    st.f32.fill_(float("nan"))
    x = tokens(9, 2, 2, 64, 64, torch.bfloat16, 5)
    parents = trees([9], "random", 2)
    o = st.step_tree(*(t.to(DEV) for t in x), i32(0, 9), i32(*parents), slots=i32(1), fresh=torch.tensor([True], device=DEV))
    want, mag = tree_ref(S, [1], [True], [0, 9], parents, *x, delta=1)
    check_tree(o, want, mag, 9, 64, torch.bfloat16, 1)


def test_tree_a_spoilt_state_row_stays_in_its_column():
    st, S = state(1, 1, 64, 64, 1)
    st.f32[0, 7, 3] = float("nan")
    st.f32[0, 9, 3] = float("inf")
    x = tokens(20, 1, 1, 64, 64, torch.bfloat16, 5)
    parents = trees([20], "random", 2)
    o = st.step_tree(*(t.to(DEV) for t in x), i32(0, 20), i32(*parents))
    want, mag = tree_ref(S, [0], None, [0, 20], parents, *x, delta=1)
    assert not bool(o[:, 0, 7].isfinite().any()) and not bool(o[:, 0, 9].isfinite().any())
    keep = [c for c in range(64) if c not in (7, 9)]
    check_tree(o[:, :, keep], want[:, :, keep], mag[:, :, keep], 20, 64, torch.bfloat16, 1)


def test_tree_refusals_on_the_device():
    """A slot beyond the handle, a tree of more than max_nodes nodes, parents that are not earlier
    nodes: NaN rows; the entry beside them is carried out."""
    counts = [5, 6, 9, 4, 4]
    cu = offsets(counts)
    n = cu[-1]
    st, S = state(4, 2, 64, 64)
    x = tokens(n, 2, 2, 64, 64, torch.float32, 6)
    parents = trees(counts, "chain", 1)
    parents[cu[3] + 2] = 2                               # itself
    parents[cu[4] + 1] = -2
    o = st.step_tree(*(t.to(DEV) for t in x), i32(*cu), i32(*parents), slots=i32(0, 4, 1, 2, 3), max_nodes=6)
    want, mag = tree_ref(S, [0], None, cu[:2], parents, *x)
    check_tree(o[:5], want[:5], mag[:5], 5, 64, torch.float32, 0)
    assert bool(o[5:].isnan().all())
    parents = trees(counts, "chain", 1)
    parents[cu[1] + 1] = 9                               # behind the tree
    o = st.step_tree(*(t.to(DEV) for t in x), i32(*cu), i32(*parents), slots=i32(0, 1, -1, -1, -1))
    assert bool(o[5:11].isnan().all()) and bool(o[:5].isfinite().all())


def test_tree_spoilt_offsets_stay_inside():
    st, S = state(4, 1, 64, 64)
    x = [t.to(DEV) for t in tokens(30, 1, 1, 64, 64, torch.float32, 7)]
    parents = i32(*([-1] * 30))
    o = st.step_tree(*x, i32(-5, 10, 4, 1 << 30), parents)
    assert bool(o[:10].isfinite().all()) and bool(o[10:].isfinite().all())
    one = st.step_tree(*(t[:10] for t in x), i32(0, 10), parents[:10])
    assert torch.equal(o[:4], one[:4])


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
def test_tree_is_step_slots_along_its_paths(io, delta, diag):
    dtype, heads, dk, dv = TYPES[io], 4, 128, 72
    st, S = state(3, heads, dk, dv, delta, diag)
    x = [t.to(DEV) for t in tokens(11, heads, 2, dk, dv, dtype, 8, diag)]
    parents = trees([11], "random", 9)
    o = st.step_tree(*x, i32(0, 11), i32(*parents), slots=i32(1))
    for leaf in (10, 9, 4):
        path = [leaf]
        while parents[path[0]] >= 0:
            path.insert(0, parents[path[0]])
        walk, _ = state(3, heads, dk, dv, delta, diag)
        for j in path:
            one = walk.step_slots(*(t[j:j + 1] for t in x), slots=i32(1))
        bound = 2 * half_step(dtype) + OPERANDS[dtype] + 64 * U32
        assert rel(o[leaf].float(), one[0].double()) <= bound


def far_rows(t, stride):
    wide = torch.zeros(((t.shape[0] - 1) * stride + t[0].numel(),), dtype=t.dtype, device=DEV)
    y = wide.as_strided(t.shape, (stride, t.shape[2], 1))
    y.copy_(t)
    return y


def test_tree_and_path_offsets_beyond_32_bits():
    """Rows and slots whose element offsets pass 2^31 (and their bytes 2^32)."""
    heads, dk, dv, n = 2, 64, 64, 18
    x = tokens(n, heads, 2, dk, dv, torch.bfloat16, 12)
    stride = (1 << 31) // (n - 2) // 8 * 8 + 8
    st, S = state(3, heads, dk, dv, 1)
    parents = trees([n], "random", 4)
    far = [far_rows(t.to(DEV), stride) if t.dim() == 3 else t.to(DEV) for t in x]
    o = st.step_tree(*far, i32(0, n), i32(*parents), slots=i32(2))
    want, mag = tree_ref(S, [2], None, [0, n], parents, *x, delta=1)
    check_tree(o, want, mag, n, dk, torch.bfloat16, 1)
    path = [0, 5, n - 1]
    st.accept_path(*far[1:], i32(0, n), torch.tensor([path], dtype=torch.int32, device=DEV), i32(3), slots=i32(2))
    pool, mag = path_ref(S, [2], None, [0, n], [path], *x[1:], delta=1)
    check_state(st, pool, mag, 3, dk, 1)
    del far
    torch.cuda.empty_cache()
    big = (1 << 31) // (heads * dk * dv) + 2             # slots
    st = lsq.LsqState(lsq.LsqConfig(batch=big, heads=heads, dk=dk, dv=dv, bits=32, group=1,
                                    policy=lsq.POLICY_NONE), device=DEV)
    last = S[0].view(heads, dv, dk).to(DEV)
    st.f32[-heads:] = last
    x = tokens(n, heads, 2, dk, dv, torch.bfloat16, 12)
    dx = [t.to(DEV) for t in x]
    o = st.step_tree(*dx, i32(0, n), i32(*parents), slots=i32(big - 1))
    want, mag = tree_ref(S[:1], [0], None, [0, n], parents, *x)
    check_tree(o, want, mag, n, dk, torch.bfloat16, 0)
    st.accept_path(*dx[1:], i32(0, n), torch.tensor([path], dtype=torch.int32, device=DEV), i32(3), slots=i32(big - 1))
    pool, mag = path_ref(S[:1], [0], None, [0, n], [path], *x[1:])
    assert rel(st.f32[-heads:].cpu(), pool[0]) <= 16 * U32


def check_state(st, pool, mag, T, dk, delta):
    S = st.f32.double().cpu().view(pool.shape)
    over = (S - pool).abs() - (3 * T + 8 + (dk if delta else 0)) * U32 * mag
    assert float(over.max()) <= 0
    assert rel(S, pool) <= (64 if delta else 16) * U32


def run_path(counts, paths, heads, qk_heads, dk, dv, dtype, delta=0, diag=0, slots=None, fresh=None, n_slots=None,
             depth=None, seed=3, pad=0):
    cu = offsets(counts)
    slots = list(range(len(counts))) if slots is None else slots
    st, S = state(n_slots or max(slots + [0]) + 2, heads, dk, dv, delta, diag)
    x = tokens(cu[-1], heads, qk_heads, dk, dv, dtype, seed, diag, False, 0)
    depth = depth or max(1, max(map(len, paths)))
    table = torch.full((len(counts), depth), 12345, dtype=torch.int32)
    for i, p in enumerate(paths):
        table[i, :len(p)] = torch.tensor(p, dtype=torch.int32)
    dx = [t.to(DEV) for t in x]
    if pad:
        dx[1:3] = [far_rows(t, t[0].numel() + pad) for t in dx[1:3]]
    got = st.accept_path(*dx[1:], i32(*cu), table.to(DEV), i32(*map(len, paths)), slots=i32(*slots),
                         fresh=None if fresh is None else torch.tensor(fresh, device=DEV))
    assert got is st
    pool, mag = path_ref(S, slots, fresh, cu, paths, *x[1:], delta=delta)
    check_state(st, pool, mag, depth, dk, delta)
    for s in range(S.shape[0]):                          # slots that no entry names, bit for bit
        if s not in slots:
            assert torch.equal(st.f32.view(S.shape)[s].cpu(), S[s])
    return st


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_path_shapes(io, delta, diag, shape):
    run_path([9, 1, 6], [[0, 2, 3, 8], [0], [5, 0]], *shape, TYPES[io], delta, diag, slots=[3, 0, 2],
             fresh=[False, True, False])


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("n", [1, 2, 3, 4, 5, 16, 17, 63, 64])
def test_path_lengths(io, n):
    run_path([70], [list(range(70 - n, 70))], 2, 1, 64, 64, TYPES[io], n % 2, 0)
    run_path([64], [list(range(n))], 1, 1, 128, 128, TYPES[io], 1 - n % 2, 1, depth=64)


@pytest.mark.parametrize("delta,diag", RULES)
def test_path_empty_padded_repeated(delta, diag):
    # nothing accepted, a padded entry, a node twice, nodes out of order, rows apart
    run_path([4, 7, 0, 5, 3], [[], [0, 0, 6, 2], [], [0, 1], [2]], 2, 2, 64, 64, torch.bfloat16, delta, diag,
             slots=[4, 1, 0, -1, 6], fresh=[True, False, False, True, True], pad=8)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
def test_path_is_step_slots_token_by_token(io, delta, diag):
    dtype, heads, dk, dv = TYPES[io], 4, 128, 72
    st, _ = state(5, heads, dk, dv, delta, diag)
    walk, _ = state(5, heads, dk, dv, delta, diag)
    x = [t.to(DEV) for t in tokens(13, heads, 2, dk, dv, dtype, 8, diag)]
    path = [0, 3, 4, 9, 12]
    st.accept_path(*x[1:], i32(0, 13), torch.tensor([path], dtype=torch.int32, device=DEV), i32(5), slots=i32(3))
    for j in path:
        walk.step_slots(*(t[j:j + 1] for t in x), slots=i32(3))
    assert torch.equal(st.f32, walk.f32)


def test_path_refusals_on_the_device():
    """A slot beyond the handle or taken, a length over the table's width, a node outside its tree:
    the state stays.  An entry with a length of zero or less takes no slot."""
    counts = [4] * 9
    cu = offsets(counts)
    st, S = state(6, 2, 64, 64)
    x = tokens(36, 2, 2, 64, 64, torch.bfloat16, 6)
    table = torch.tensor([[0, 1], [0, 1], [0, 4], [0, -1], [0, 1], [0, 1], [0, 1], [0, 3], [1, 1]], dtype=torch.int32)
    lengths = [0, 2, 2, 2, 3, 2, -1, 2, 2]
    slots = [0, 0, 1, 2, 3, 6, 4, 4, 0]                  # entry 8: slot 0, which entry 1 takes
    st.accept_path(*(t.to(DEV) for t in x[1:]), i32(*cu), table.to(DEV), i32(*lengths), slots=i32(*slots))
    pool, mag = path_ref(S, [-1, 0, -1, -1, -1, -1, -1, 4], None, cu, [[], [0, 1], [], [], [], [], [], [0, 3]], *x[1:])
    check_state(st, pool, mag, 2, 64, 0)
    for s in (1, 2, 3, 5):
        assert torch.equal(st.f32.view(S.shape)[s].cpu(), S[s])
    # nothing but NaN: a path of no columns, entries of no nodes
    before = st.f32.clone()
    st.accept_path(*(t.to(DEV) for t in x[1:]), i32(*cu), table[:, :0].to(DEV).contiguous(), i32(*lengths), slots=i32(*slots))
    st.accept_path(*(t.to(DEV) for t in x[1:]), i32(*[0] * 10), table.to(DEV), i32(*[1] * 9), slots=i32(*slots))
    assert torch.equal(st.f32, before)


def test_path_fresh_ignores_a_spoilt_slot():
    st, S = state(2, 2, 64, 64, 1)
    st.f32.view(2, 2, 64, 64)[1] = float("nan")
    x = tokens(3, 2, 2, 64, 64, torch.bfloat16, 5)
    st.accept_path(*(t.to(DEV) for t in x[1:]), i32(0, 3), torch.tensor([[0, 2]], dtype=torch.int32, device=DEV),
                   i32(2), slots=i32(1), fresh=torch.tensor([True], device=DEV))
    pool, mag = path_ref(S, [1], [True], [0, 3], [[0, 2]], *x[1:], delta=1)
    check_state(st, pool, mag, 2, 64, 1)


# ---- verification ------------------------------------------------------------------------------

def drafts(counts, vocab, shape, seed, drawn, sharp=2.0, error=0.7):
    """Rows, tokens and uniform numbers of packed trees (CPU)."""
    g = torch.Generator().manual_seed(seed)
    n = sum(counts)
    logits = sharp * torch.randn((n, vocab), generator=g)
    target = logits.softmax(-1)
    logits = logits + error * torch.randn((n, vocab), generator=g)
    draft = logits.softmax(-1)
    parents, cu = trees(counts, shape, seed), offsets(counts)
    ids = torch.zeros(n, dtype=torch.int32)
    for i, c in enumerate(counts):
        used = {}
        for j in range(c):
            p = parents[cu[i] + j]
            if p < 0:
                continue
            row = draft[cu[i] + p].clone()
            if drawn != "with":
                row[used.setdefault(p, [])] = 0.0
            if float(row.sum()) == 0.0:                  # more children than tokens
                row += 1.0
            ids[cu[i] + j] = int(torch.multinomial(row, 1, generator=g))
            used.setdefault(p, []).append(int(ids[cu[i] + j]))
    return dict(target=target, draft=None if drawn == "given" else draft, ids=ids, parents=parents, cu=cu,
                uniform=torch.rand(n, generator=g), uniform_next=torch.rand(len(counts), generator=g))


def run_verify(d, drawn, depth=64, stride=0, base=0):
    def rows(t):
        if t is None or not stride:
            return None if t is None else t.to(DEV)
        wide = torch.full((t.shape[0] * (t.shape[1] + stride) + base,), float("nan"), device=DEV)
        y = wide[base:].view(t.shape[0], -1)[:, :t.shape[1]]
        y.copy_(t)
        return y
    path, lengths, token = lsq.verify_tree(rows(d["target"]), d["ids"].to(DEV), i32(*d["parents"]), i32(*d["cu"]),
                                           d["uniform"].to(DEV), d["uniform_next"].to(DEV), draft=rows(d["draft"]),
                                           replacement=drawn == "with", depth=depth)
    return path.tolist(), lengths.tolist(), token.tolist()


def check_verify(d, drawn, depth=64, **kw):
    got = run_verify(d, drawn, depth, **kw)
    want = verify_ref(d["target"], d["draft"], d["ids"], d["parents"], d["cu"], d["uniform"], d["uniform_next"],
                      drawn == "with", depth)
    assert got == tuple(want)
    return got


DRAWN = ["with", "without", "given"]


@pytest.mark.parametrize("drawn", DRAWN)
@pytest.mark.parametrize("vocab", [1, 2, 3, 5, 63, 64, 65, 1000, 4095, 4096, 4097, 8191, 20011, 131072, 262145])
def test_verify_vocabularies(drawn, vocab):
    counts = [5, 1, 12, 0, 9] if vocab > 10000 else [5, 1, 33, 0, 64, 9, 17]
    rejected = 0
    for seed in (1, 2):
        d = drafts(counts, vocab, "random" if seed == 1 else "star", seed, drawn)
        for i, a in enumerate(d["cu"][:-1]):
            if counts[i]:
                d["parents"][a] = -1
        path, lengths, token = check_verify(d, drawn)
        rejected += sum(n < c for n, c in zip(lengths, counts))
    assert rejected or vocab < 4


@pytest.mark.parametrize("drawn", DRAWN)
@pytest.mark.parametrize("kind", ["chain", "star", "forest", "random"])
@pytest.mark.parametrize("n", [1, 2, 16, 63, 64])
def test_verify_trees(drawn, kind, n):
    for seed in range(4):
        d = drafts([n] * 6, 501, kind, 10 * seed + n, drawn, error=0.3 if seed % 2 else 1.5)
        check_verify(d, drawn, depth=(64, 1, 3, n)[seed])


@pytest.mark.parametrize("drawn", DRAWN)
def test_verify_rows_apart_and_unaligned(drawn):
    for stride, base in ((1, 0), (3, 1), (61, 2), (4, 3)):
        d = drafts([9, 20], 5003, "random", 3, drawn)
        check_verify(d, drawn, stride=stride, base=base)


@pytest.mark.parametrize("drawn", DRAWN)
def test_verify_at_exact_borders(drawn):
    """Probabilities and numbers that are multiples of powers of two: every sum is exact, ties fall on
    the border itself (a child is taken if less, the next token is the first that exceeds)."""
    V = 8192
    g = torch.Generator().manual_seed(7)
    for seed in range(6):
        d = drafts([4, 7, 1], V, "star", seed, drawn)
        n = d["target"].shape[0]
        for name in ("target", "draft"):
            if d[name] is not None:
                w = torch.randint(0, 3, (n, V), generator=g).float()
                w[:, -1] = 0
                w[:, 0] = 2 * V - w[:, 1:].sum(-1)        # every row sums to 2 V / (2 V)
                d[name] = w / (2 * V)
        d["uniform"] = torch.randint(0, 2, (n,), generator=g).float() / 2
        d["uniform_next"] = torch.randint(0, V, (3,), generator=g).float() / V
        got = run_verify(d, drawn)
        want = verify_ref(d["target"], d["draft"], d["ids"], d["parents"], d["cu"], d["uniform"], d["uniform_next"],
                          drawn == "with", 64)
        # where the walk ends at an untouched row (one node, or a leaf) its sums are exact in any order
        for i, n_i in enumerate(got[1]):
            assert got[0][i] == want[0][i] and got[1][i] == want[1][i]
            if i == 2 or n_i == 2:
                assert got[2][i] == want[2][i]


def test_verify_equal_rows_accept_everything():
    # p = q: the ratio is one, every first child is taken
    d = drafts([8, 20], 3001, "chain", 4, "with")
    d["draft"] = d["target"].clone()
    path, lengths, token = check_verify(d, "with")
    assert lengths == [8, 20]
    # uniform 0 takes any child with a probability, however small; none without
    d = drafts([3], 100, "star", 4, "with")
    d["uniform"].zero_()
    assert run_verify(d, "with")[1] == [2]
    d["target"][0] = 0.0
    d["target"][0, 50] = 1.0
    d["ids"][:] = torch.tensor([0, 7, 50])
    path, lengths, token = run_verify(d, "with")
    assert path[0][:2] == [0, 2]


def test_verify_least_and_largest_numbers():
    d = drafts([1, 1], 1000, "chain", 4, "with")
    d["target"][:, :10] = 0.0
    d["target"][:, -7:] = 0.0
    d["uniform_next"][0] = 0.0
    d["uniform_next"][1] = 1.0                           # out of the range: the last with a probability
    assert run_verify(d, "with")[2] == [10, 992]
    d["uniform_next"][:] = torch.tensor([float("nan"), -3.0])
    assert run_verify(d, "with")[2] == [10, 10]


@pytest.mark.parametrize("drawn", DRAWN)
def test_verify_passes_over_bad_tokens_and_nan(drawn):
    d = drafts([6, 6], 300, "star", 4, drawn)
    d["ids"][1] = -1
    d["ids"][2] = 300
    d["ids"][8] = 2 ** 31 - 1
    check_verify(d, drawn)
    # NaN counts as no probability: as if it were 0
    d = drafts([6, 6], 5000, "star", 5, drawn)
    clean = {**d, "target": d["target"].clone()}
    clean["target"][:, 17] = clean["target"][:, 4500] = 0.0
    d["target"][:, 17] = d["target"][:, 4500] = float("nan")
    assert run_verify(d, drawn) == run_verify(clean, drawn)


def test_verify_rows_without_mass():
    d = drafts([1, 2], 300, "chain", 4, "with")
    d["target"].zero_()
    assert run_verify(d, "with")[1:] == ([1, 1], [-1, -1])
    # p = q up to one token that is drawn and fails: nothing is left, the token comes from p
    d = drafts([2], 4, "chain", 4, "with")
    d["target"][0] = torch.tensor([0.25, 0.25, 0.25, 0.0])
    d["draft"][0] = torch.tensor([0.25, 0.25, 0.25, 0.25])
    d["ids"][1] = 3
    d["uniform_next"][0] = 0.5
    path, lengths, token = run_verify(d, "with")
    assert (lengths, token) == ([1], [1])
    # every token given and none taken: the same
    d = drafts([3], 2, "star", 4, "given")
    d["target"][0] = torch.tensor([0.0, 0.0])
    d["ids"][1:] = torch.tensor([0, 1])
    assert run_verify(d, "given")[1:] == ([1], [-1])


def test_verify_the_same_token_twice():
    for drawn in DRAWN:
        for seed in range(8):
            d = drafts([5, 5, 5, 5], 12, "star", seed, drawn, error=2.0)
            d["ids"][2] = d["ids"][1]
            d["ids"][13] = d["ids"][11]
            if drawn == "without":                       # only with draws that are worth something
                d["draft"] = d["draft"] * 0.4
            check_verify(d, drawn)


def test_verify_refusals_on_the_device():
    d = drafts([3, 65, 3, 0, 3], 300, "chain", 4, "with")
    d["parents"][d["cu"][2] + 1] = 1
    d["parents"][d["cu"][4] + 2] = -2
    path, lengths, token = run_verify(d, "with", depth=70)
    assert lengths[1:] == [0] * 4 and token[1:] == [-1] * 4
    assert all(x == [-1] * 70 for x in path[1:])
    assert lengths[0] >= 1 and path[0][0] == 0 and 0 <= token[0] < 300
    d["cu"] = [-4, 3, 1, 1 << 30]                        # clamped: [0, 3), empty, too many
    path, lengths, token = run_verify({**d, "uniform_next": d["uniform_next"][:3]}, "with")
    assert lengths[1:] == [0, 0] and lengths[0] >= 1


def test_verify_offsets_beyond_32_bits():
    vocab, n = 1000, 6
    d = drafts([n], vocab, "random", 3, "without")
    d["parents"][0] = -1
    stride = (1 << 31) // (n - 1) + 4
    far = []
    for name in ("target", "draft"):
        wide = torch.zeros((n - 1) * stride + vocab, device=DEV)
        y = wide.as_strided((n, vocab), (stride, 1))
        y.copy_(d[name])
        far.append(y)
    path, lengths, token = lsq.verify_tree(far[0], d["ids"].to(DEV), i32(*d["parents"]), i32(0, n),
                                           d["uniform"].to(DEV), d["uniform_next"].to(DEV), draft=far[1], replacement=False)
    want = verify_ref(d["target"], d["draft"], d["ids"], d["parents"], d["cu"], d["uniform"], d["uniform_next"], False, 64)
    assert (path.tolist(), lengths.tolist(), token.tolist()) == tuple(want)


# ---- together ----------------------------------------------------------------------------------

def test_a_run_of_drafted_decoding():
    """As a serving program makes it: prompts, then rounds of trees whose outputs make the target's
    rows, their verification, and the accepted tokens written into the slots.  The slots end where
    the accepted tokens alone, step by step, would have brought them."""
    heads, hk, dk, dv, vocab, dtype = 4, 2, 128, 64, 600, torch.bfloat16
    g = torch.Generator().manual_seed(3)
    table = {x: torch.randn((vocab, h, d), generator=g) / d ** 0.5 for x, h, d in
             (("q", hk, dk), ("k", hk, dk), ("v", heads, dv))}
    table = {x: t.to(dtype).to(DEV) for x, t in table.items()}
    gate = torch.sigmoid(torch.randn((vocab, heads), generator=g) + 2).to(DEV)
    write = torch.sigmoid(torch.randn((vocab, heads), generator=g)).to(DEV)
    head = (torch.randn((heads * dv, vocab), generator=g) * 1.5).to(DEV)

    def inputs(ids):
        at = ids.long()
        return table["q"][at], table["k"][at], table["v"][at], gate[at].contiguous(), write[at].contiguous()

    pool, _ = state(6, heads, dk, dv, 1)
    plain, _ = state(6, heads, dk, dv, 1)
    slots = i32(4, 0, 3)
    prompt = torch.randint(0, vocab, (30,), generator=g).to(DEV)
    for st in (pool, plain):
        st.attend(*inputs(prompt), i32(0, 12, 20, 30), slots=slots, fresh=torch.ones(3, dtype=torch.bool, device=DEV))
    pending = torch.randint(0, vocab, (3,), generator=g).to(torch.int32).to(DEV)
    moved = 0
    for step in range(6):
        counts = [9, 1, 6]
        cu = offsets(counts)
        parents = trees(counts, "random", step)
        for a, c in zip(cu, counts):
            parents[a] = -1
            parents[a + 1:a + c] = [max(0, p) for p in parents[a + 1:a + c]]
        ids = torch.randint(0, vocab, (16,), generator=g).to(torch.int32).to(DEV)
        ids[cu[:-1]] = pending
        x = inputs(ids)
        o = pool.step_tree(*x, i32(*cu), i32(*parents), slots=slots, max_nodes=9)
        target = (o.float().flatten(1) @ head).softmax(-1)
        # drafts with a fair chance: each node's token is among its parent's likelier ones
        draft = (target + 1.0 / vocab) / 2
        best = target.topk(9, -1).indices.to(torch.int32)
        for a, c in zip(cu, counts):
            for j in range(1, c):
                ids[a + j] = best[a + parents[a + j], j % 3]
        x = inputs(ids)                                  # rows of the drafted tokens; node 0's stay
        o = pool.step_tree(*x, i32(*cu), i32(*parents), slots=slots, max_nodes=9)
        target = (o.float().flatten(1) @ head).softmax(-1)
        uniform, last = torch.rand(16, generator=g), torch.rand(3, generator=g)
        path, lengths, token = lsq.verify_tree(target, ids, i32(*parents), i32(*cu), uniform.to(DEV), last.to(DEV),
                                               draft=draft.contiguous(), depth=6)
        want = verify_ref(target.cpu(), draft.cpu(), ids.cpu(), parents, cu, uniform, last, True, 6)
        assert (path.tolist(), lengths.tolist(), token.tolist()) == tuple(want)
        pool.accept_path(*x[1:], i32(*cu), path, lengths, slots=slots)
        for i in range(3):                               # token by token on the other handle
            for j in path[i, :lengths[i]].tolist():
                at = cu[i] + j
                plain.step_slots(*(t[at:at + 1] for t in x), slots=slots[i:i + 1])
        assert torch.equal(pool.f32, plain.f32)
        moved += int(lengths.sum()) - 3
        pending = token
    assert moved > 0


# ---- streams, graphs, batches ------------------------------------------------------------------

def _tree_case(seed=1, delta=1):
    counts = [9, 17, 3]
    cu = offsets(counts)
    x = [t.to(DEV) for t in tokens(cu[-1], 4, 2, 128, 128, torch.bfloat16, seed)]
    return x, i32(*cu), i32(*trees(counts, "random", seed)), counts


def test_replayed_graphs_take_other_slots_trees_and_paths():
    """One captured run of tree, verification and acceptance, replayed with other contents in the same
    buffers and eager work between: every replay is what eager calls give."""
    vocab, dk = 70001, 128
    st, _ = state(6, 4, dk, 128, 1)
    ref, _ = state(6, 4, dk, 128, 1)
    x, cu, parents, counts = _tree_case()
    slots, fresh = i32(4, 0, 2), torch.tensor([False, True, False], device=DEV)
    d = drafts(counts, vocab, "random", 1, "with")
    rows = {n: d[n].to(DEV) for n in ("target", "draft", "ids", "uniform", "uniform_next")}
    tree = i32(*d["parents"])

    def run(s):
        o = s.step_tree(*x, cu, parents, slots=slots, fresh=fresh, max_nodes=32)
        path, lengths, token = lsq.verify_tree(rows["target"], rows["ids"], tree, cu, rows["uniform"],
                                               rows["uniform_next"], draft=rows["draft"], depth=8)
        s.accept_path(*x[1:], cu, path, lengths, slots=slots, fresh=fresh)
        return o, path, lengths, token

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run(st)
    torch.cuda.current_stream().wait_stream(stream)
    st.f32.copy_(ref.f32)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = run(st)
    st.f32.copy_(ref.f32)
    for step in range(4):
        y, _, p, _ = _tree_case(seed=10 + step)
        for a, b in zip(x, y):
            a.copy_(b)
        parents.copy_(p)
        e = drafts(counts, vocab, "random", 20 + step, "with")
        for n in rows:
            rows[n].copy_(e[n])
        tree.copy_(i32(*e["parents"]))
        slots.copy_(i32(*[(4, 0, 2), (5, 1, 3), (0, -1, 5), (2, 2, 1)][step]))
        g.replay()
        got = [t.clone() for t in out]
        torch.cuda.synchronize()
        want = run(ref)                                  # eager, on another handle
        named = [i for i in range(3) if int(slots[i]) >= 0]
        begin = offsets(counts)
        for i in named:
            assert torch.equal(got[0][begin[i]:begin[i + 1]], want[0][begin[i]:begin[i + 1]])
        for a, b in zip(got[1:], want[1:]):
            assert torch.equal(a, b)
        assert torch.equal(st.f32, ref.f32)


def test_calls_on_other_streams():
    """Two streams at once, each with a handle and a batch of its own."""
    runs = []
    for seed in (1, 2):
        st, _ = state(4, 4, 128, 128, 1, seed=seed)
        x, cu, parents, counts = _tree_case(seed)
        d = drafts(counts, 70001, "random", seed, "without")
        rows = [d[n].to(DEV) for n in ("target", "ids", "uniform", "uniform_next", "draft")]
        runs.append((st, x, cu, parents, rows, i32(*d["parents"]), torch.cuda.Stream()))
    torch.cuda.synchronize()

    def run(st, x, cu, parents, rows, tree, stream, given):
        kw = dict(stream=stream if given else None)
        o = st.step_tree(*x, cu, parents, slots=i3, max_nodes=17, **kw)
        v = lsq.verify_tree(rows[0], rows[1], tree, cu, rows[2], rows[3], draft=rows[4], replacement=False, depth=9, **kw)
        st.accept_path(*x[1:], cu, v[0], v[1], slots=i3, **kw)
        return o, *v, st.f32.clone() if not given else None

    i3 = i32(3, 0, 2)
    before = [r[0].f32.clone() for r in runs]
    torch.cuda.synchronize()
    got = [run(*r, True) for _ in range(1) for r in runs]
    torch.cuda.synchronize()
    states = [r[0].f32.clone() for r in runs]
    for r, b, g, s in zip(runs, before, got, states):
        r[0].f32.copy_(b)
        want = run(*r, False)
        for a, w in zip(g[:4], want[:4]):
            assert torch.equal(a, w)
        assert torch.equal(s, want[4])


def test_the_same_call_gives_the_same_bits():
    st, _ = state(4, 4, 128, 128, 1)
    x, cu, parents, counts = _tree_case()
    first = st.step_tree(*x, cu, parents)
    for _ in range(5):
        assert torch.equal(st.step_tree(*x, cu, parents), first)


def test_fewer_nodes_than_max_nodes_allows():
    # the bound chooses the kernel's size, not its results beyond rounding
    st, S = state(4, 4, 128, 128, 1)
    x, cu, parents, counts = _tree_case()
    want, mag = tree_ref(S, [0, 1, 2], None, cu.tolist(), parents.tolist(), *(t.cpu() for t in x), delta=1)
    for bound in (17, 32, 33, 48, 64):
        o = st.step_tree(*x, cu, parents, max_nodes=bound)
        check_tree(o, want, mag, 17, 128, torch.bfloat16, 1)


def test_verify_many_entries():
    counts = [(5 * i) % 7 + 1 for i in range(300)]
    d = drafts(counts, 700, "random", 2, "without")
    for a in d["cu"][:-1]:
        d["parents"][a] = -1
    check_verify(d, "without", depth=5)


@pytest.mark.parametrize("drawn", DRAWN)
@pytest.mark.parametrize("counts", [[1, 2, 0], [7, 8], [9, 10, 1, 17], [16, 17, 20]], ids=str)
def test_verify_several_sums(drawn, counts):
    """Large rows of trees of several sizes, where most children are rejected: sums by launches of their
    own, fewer and more than the entries need."""
    most = 0
    for seed, vocab in ((1, 70001), (2, 140000)):
        d = drafts(counts, vocab, "star" if seed == 1 else "random", seed, drawn, error=2.5)
        for a, c in zip(d["cu"], counts):
            if c:
                d["parents"][a] = -1
                d["parents"][a + 1:a + c] = [max(0, p) for p in d["parents"][a + 1:a + c]]
        lengths = check_verify(d, drawn, depth=5)[1]
        most = max(most, max(c - n for c, n in zip(counts, lengths)))
    assert most >= max(counts) // 3                      # nodes that were not accepted


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
def test_tree_fast_and_slow_decays(io, delta, diag):
    # products of decays that leave the range of fp32, and decays so near one that their logarithms matter
    for power in (40.0, 1e-4):
        def edit(x):
            x["alpha"].pow_(power)
        for kind in ("chain", "random"):
            o, want, mag, T = run_tree([40], kind, 2, 1, 64, 64, TYPES[io], delta, diag, edit=edit)
            check_tree(o, want, mag, T, 64, TYPES[io], delta)


@pytest.mark.parametrize("io", TYPES)
def test_tree_and_path_broadcast_rows(io):
    # one row of q, k, v for all nodes (stride 0)
    dtype, n = TYPES[io], 21
    st, S = state(2, 4, 128, 72, 1)
    x = list(tokens(n, 4, 2, 128, 72, dtype, 8))
    x[:3] = [t[:1].expand_as(t) for t in x[:3]]
    dx = [t.to(DEV) for t in x]
    dx[:3] = [t[:1].to(DEV).expand(t.shape) for t in x[:3]]
    parents = trees([n], "random", 6)
    o = st.step_tree(*dx, i32(0, n), i32(*parents), slots=i32(1), max_nodes=21)
    want, mag = tree_ref(S, [1], None, [0, n], parents, *x, delta=1)
    check_tree(o, want, mag, n, 128, dtype, 1)
    path = [0, 4, 20]
    st.accept_path(*dx[1:], i32(0, n), torch.tensor([path], dtype=torch.int32, device=DEV), i32(3), slots=i32(1))
    pool, mag = path_ref(S, [1], None, [0, n], [path], *x[1:], delta=1)
    check_state(st, pool, mag, 3, 128, 1)


def test_tree_without_a_bound_or_slots():
    # max_nodes left to its default, slots to the entries' order; many value heads to a key head, an odd count
    counts = [3, 30, 64, 1]
    for heads, hk in ((5, 1), (16, 2), (7, 7)):
        cu = offsets(counts)
        st, S = state(4, heads, 64, 48, 1)
        x = tokens(cu[-1], heads, hk, 64, 48, torch.bfloat16, 8)
        parents = trees(counts, "random", 6)
        o = st.step_tree(*(t.to(DEV) for t in x), i32(*cu), i32(*parents))
        want, mag = tree_ref(S, [0, 1, 2, 3], None, cu, parents, *x, delta=1)
        check_tree(o, want, mag, 64, 64, torch.bfloat16, 1)


def test_states_of_large_and_small_magnitudes():
    for scale in (2.0 ** 100, 2.0 ** -80):
        for io in ("bf16", "f32"):
            st, S = state(1, 2, 64, 64, 0, scale=scale)
            x = list(tokens(20, 2, 2, 64, 64, TYPES[io], 8))
            x[2] = (x[2].float() * scale).to(TYPES[io])
            parents = trees([20], "random", 6)
            o = st.step_tree(*(t.to(DEV) for t in x), i32(0, 20), i32(*parents))
            want, mag = tree_ref(S, [0], None, [0, 20], parents, *x)
            check_tree(o, want, mag, 20, 64, TYPES[io], 0)
