"""How far step_tree may be off where an output's terms cancel: operands keep 24 bits whatever the
input's type (GPU).

Each case has at most three terms that are not zero, with A the sum of their magnitudes.  An operand
of three bf16 parts is off by 2^-27 of itself, the three products of parts left out are 2^-26 of theirs,
and what is made in fp32 (a decay's product, a gate, a write, at most six products of parts per sum, added
one by one) takes at most twelve roundings of u = 2^-24: 16 u A in all, beside the output's own half
step.  Operands of two parts (16 bits) miss up to 2^-17 of a value in [1, 2), half of that 32 u, on most
of the values tried here.
"""
import pytest
import torch

from tests.drafts_ref import tree_ref
from tests.slots_ref import U32, half_step
from tests.test_gpu_drafts import DEV, RULES, TYPES, i32, offsets
from tests.test_gpu_slots import state

pytestmark = pytest.mark.gpu
HEADS = 8


def rounded(x, bits):
    """x in [1, 2) to so many bits behind the point."""
    return (x * 2.0 ** bits).round() / 2.0 ** bits


def draws(*shape, seed=1):
    return 1 + torch.rand(shape, generator=torch.Generator().manual_seed(seed))


def blank(n, dk, dv, diag):
    """Nodes that neither decay, write nor read."""
    alpha = torch.ones((n, HEADS, dk) if diag else (n, HEADS))
    return [torch.zeros(n, HEADS, dk), torch.zeros(n, HEADS, dk), torch.zeros(n, HEADS, dv), alpha, torch.zeros(n, HEADS)]


def check(io, S, fresh, x, n, dk, dv, delta, diag, max_nodes):
    dtype = TYPES[io]
    st, _ = state(1, HEADS, dk, dv, delta, diag)
    st.f32.copy_(S.view(st.f32.shape))
    x = [t.to(dtype) for t in x[:3]] + x[3:]
    parents = list(range(-1, n - 1))
    o = st.step_tree(*(t.to(DEV) for t in x), i32(0, n), i32(*parents), fresh=torch.tensor([fresh], device=DEV),
                     max_nodes=max_nodes).double().cpu()
    want, mag = tree_ref(S, [0], [fresh], offsets([n]), parents, *x, delta=delta)
    lost = 16 * U32 * mag
    bound = lost + half_step(dtype) * (want.abs() + lost) + (2.0 ** -25 if io == "f16" else 0.0)
    over = (o - want).abs() - bound
    assert float(over.max()) <= 0, f"off by {float(over.max())} over the bound"
    last = want[-1].abs() / mag[-1]
    assert 0 < float(last.max()) < 2.0 ** -10            # the terms do cancel


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
@pytest.mark.parametrize("n", [1, 16, 17, 40, 64])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 72), (128, 64), (128, 128)])
def test_a_state_whose_products_cancel(io, delta, diag, n, dk, dv):
    S = torch.zeros(1, HEADS, dv, dk)
    S[..., 0] = draws(HEADS, dv)
    S[..., 1] = -rounded(S[..., 0], 12)
    x = blank(n, dk, dv, diag)
    x[0][:, :, :2] = 1
    check(io, S, False, x, n, dk, dv, delta, diag, n)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", RULES)
@pytest.mark.parametrize("n", [2, 16, 17, 40, 64])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 72), (128, 64), (128, 128)])
def test_writes_that_cancel(io, delta, diag, n, dk, dv):
    # two writes into columns of their own, with gates of 24 and of 12 bits
    x = blank(n, dk, dv, diag)
    x[0][-1, :, :2] = 1
    x[1][0, :, 0] = x[1][-1, :, 1] = 1
    x[2][0] = rounded(draws(HEADS, dv, seed=2), 7)
    x[2][-1] = -x[2][0]
    x[4][0] = draws(HEADS, seed=3)
    x[4][-1] = rounded(x[4][0], 12)
    check(io, torch.zeros(1, HEADS, dv, dk), True, x, n, dk, dv, delta, diag, n)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("diag", [0, 1])
@pytest.mark.parametrize("n", [2, 16, 17, 40, 64])
@pytest.mark.parametrize("dk,dv", [(64, 64), (64, 72), (128, 64), (128, 128)])
def test_scores_that_cancel(io, diag, n, dk, dv):
    # q.k of two nodes, of up to 16 bits and apart by one bit of a small factor
    x = blank(n, dk, dv, diag)
    c, a, b = (rounded(draws(HEADS, seed=s), 7) for s in (4, 5, 6))
    b = torch.where(b > 1.5, 1.5 - 2.0 ** -7, b)
    x[0][-1, :, 0], x[0][-1, :, 1] = 1, a * 2.0 ** -4
    x[1][0, :, 0], x[1][0, :, 1] = c, b * 2.0 ** -5
    x[1][-1, :, 0], x[1][-1, :, 1] = c, (b + 2.0 ** -7) * 2.0 ** -5
    x[2][0], x[2][-1] = 1, -1
    x[4].fill_(1)
    check(io, torch.zeros(1, HEADS, dv, dk), True, x, n, dk, dv, 0, diag, n)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta", [0, 1])
@pytest.mark.parametrize("n", [1, 16, 17, 40, 64])
def test_decays_of_channels_that_cancel(io, delta, n, dk=128, dv=128):
    S = torch.ones(1, HEADS, dv, dk)
    x = blank(n, dk, dv, 1)
    x[3][0, :, 0] = draws(HEADS, seed=7) / 2
    S[..., 1] = -rounded(x[3][0, :, 0], 12)[None, :, None]
    x[0][:, :, :2] = 1
    check(io, S, False, x, n, dk, dv, delta, 1, n)
