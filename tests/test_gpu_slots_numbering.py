"""attend over batches that fill the GPU (GPU): how workgroups find their sequence, segment and row.

Batches of more workgroups than CUs are numbered by length, up to 64 sequences at a time, and long
sequences are cut into segments; a wrong number would skip a sequence or take one twice.  Slots are
permuted; one entry is padded, one names a slot beyond the handle and one a slot taken before.

Tolerances (fixed before the first run).  u = 2^-24, B the output's terms by their absolute values,
A the state's.  fp32 sums: (3 T + Dk + 16) u B of an output after T tokens, (3 T + 8) u A of the
state (a decay, a gate and a write per token, 8 u for the decays' logarithms and exponentials).  A
16-bit output's operands are sums of two bf16 parts, so a bf16 output lacks 2^-16 B at most (the
state's, or P's, third part), a binary16 one 3 * 2^-16 B (P: the product of the second parts of q
and k, its own third part, the product of its second part with v's); it is then rounded once, half
a step.
"""
import pytest
import torch

from tests.slots_ref import U32, batch_ref, half_step, rel, tokens
from tests.test_gpu_slots import DEV, TYPES, offsets, state

pytestmark = pytest.mark.gpu
PARTS = {"bf16": 2.0 ** -16, "f16": 3 * 2.0 ** -16, "f32": 0.0}


def check(io, lens, heads, qk_heads, dk, dv, slots=None, n_slots=None, seed=90):
    """attend against 64 bits; entries whose slot is beyond the handle or taken are refused."""
    dtype, cu = TYPES[io], offsets(lens)
    slots = list(range(len(lens))) if slots is None else slots
    n_slots = n_slots or max(slots) + 1
    fresh = [i % 3 == 1 for i in range(len(lens))]
    st, S = state(n_slots, heads, dk, dv)
    x = tokens(cu[-1], heads, qk_heads, dk, dv, dtype, seed)
    i32 = lambda y: torch.tensor(y, dtype=torch.int32, device=DEV)
    o = torch.full((cu[-1], heads, dv), 7.0, dtype=dtype, device=DEV)
    args = [y.to(DEV) for y in x]
    st.attend(*args, i32(cu), slots=i32(slots), fresh=torch.tensor(fresh, device=DEV), o=o)
    does, seen = [], set()
    for n, s in zip(lens, slots):
        ok = 0 <= s < n_slots and s not in seen
        does.append(s if ok else -1)
        if ok and n:
            seen.add(s)
    want, pool, ao, mag = batch_ref(S, does, fresh, cu, *x)
    got, T = o.double().cpu(), max(lens)
    for i, s in enumerate(slots):
        rows = got[cu[i]:cu[i + 1]]
        if does[i] < 0:
            assert bool((rows == 7.0).all() if s < 0 else rows.isnan().all()), f"entry {i}"
    live = ~want.isnan()
    assert bool(got[live].isfinite().all())
    bound = half_step(dtype) * want.abs() + ((3 * T + dk + 16) * U32 + PARTS[io]) * ao * (1 + half_step(dtype))
    if io == "f16":
        bound = bound + 2.0 ** -25               # half a step of a subnormal
    assert float(((got - want).abs() - bound)[live].max()) <= 0
    assert rel(got[live], want[live]) <= half_step(dtype) + PARTS[io] + 16 * U32
    Sg = st.f32.double().cpu().view(pool.shape)
    assert float(((Sg - pool).abs() - (3 * T + 8) * U32 * mag).max()) <= 0
    assert rel(Sg, pool) <= 16 * U32
    return st, S, args, i32(cu), i32(slots), torch.tensor(fresh, device=DEV), o


def ragged(n, most):
    """n lengths from 0 to most, empty ones among them."""
    return [0 if i % 7 == 3 else 1 + (i * 13) % most for i in range(n)]


def spoilt(n, n_slots):
    """Permuted slots, with a padded entry, one beyond the handle and one named before."""
    s = [(5 * i + 2) % n_slots for i in range(n)]
    s[1], s[n - 2], s[n - 1] = -1, n_slots, s[0]
    return s


# Workgroups: 640 and more on 256 CUs; rows of a sequence that divide by eight and by 256, by eight
# alone, by neither; more than 64 sequences.  Dk 128 in fp32 holds one workgroup per CU, others two.
@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("heads,qk_heads", [(32, 4), (24, 24), (20, 5), (9, 1)])
@pytest.mark.parametrize("seqs", [20, 64, 65, 130])
def test_whole_sequences_by_length(io, heads, qk_heads, seqs):
    check(io, ragged(seqs, 45), heads, qk_heads, 64, 16, spoilt(seqs, 131), 131)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("heads,dv,seqs", [(32, 8, 20), (24, 4, 30), (33, 5, 12), (300, 2, 4), (8, 136, 40)])
def test_whole_sequences_of_wide_rows(io, heads, dv, seqs):
    check(io, ragged(seqs, 40), heads, 1, 128, dv, spoilt(seqs, 47), 47)


# Cut sequences beside short ones: rows that divide by eight, and not; more segments than a round of
# 256 workgroups holds (8 rows: 32 segments of 256 tokens); more than 64 sequences.
@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("lens,heads,dk,dv", [([30, 2100, 0, 3000, 700], 8, 64, 16), ([2100, 1, 3000], 6, 64, 8),
                                              ([5100, 40, 4300], 8, 64, 4), ([2400, 0, 2500], 8, 128, 4),
                                              ([2700] + [0, 9, 33] * 24 + [1900, 5], 2, 64, 16)], ids=str)
def test_cut_sequences(io, lens, heads, dk, dv):
    n = len(lens)
    st, S, args, cu, slots, fresh, o = check(io, lens, heads, 2, dk, dv, [(5 * i + 2) % (n + 4) for i in range(n)]
                                             if (n + 4) % 5 else list(range(n)), n + 4)
    # the same batch gives the same bits on every call
    first = o.clone(), st.f32.clone()
    for _ in range(3):
        st.f32.copy_(S.view(st.f32.shape))
        again = st.attend(*args, cu, slots=slots, fresh=fresh)
        assert torch.equal(again, first[0]) and torch.equal(st.f32, first[1])


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("dk,dv", [(64, 201), (128, 256), (64, 300), (128, 385)])
def test_several_slices_of_columns(io, dk, dv):
    check(io, [40, 1, 75], 2, 1, dk, dv, [2, 0, 1])
