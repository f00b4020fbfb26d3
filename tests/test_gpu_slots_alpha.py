"""Decays outside (2^-126, 1] where tokens are walked one by one (GPU): the delta rule, a diagonal
decay, and single tokens of any handle multiply by them as they stand.

Tolerance as in test_gpu_slots: with signs that mix, 64 u in the 2-norm (u = 2^-24; a state element
has 3 roundings per token and, under the delta rule, those of a sum of Dk = 64 terms).
"""
import pytest
import torch

from tests.slots_ref import U32, recur, rel, tokens
from tests.test_gpu_slots import DEV, state

pytestmark = pytest.mark.gpu
N, AT, HEADS, DK, DV = 12, 5, 3, 64, 40
WALKED = [("attend", 1, 0), ("attend", 0, 1), ("attend", 1, 1), ("step", 0, 0), ("step", 1, 0), ("step", 0, 1)]


def run(st, how, x):
    """All tokens of one sequence in slot 0: (o, S [heads, dv, dk])."""
    x = [y.to(DEV) for y in x]
    if how == "attend":
        o = st.attend(*x, torch.tensor([0, N], dtype=torch.int32, device=DEV))
    else:
        o = torch.cat([st.step_slots(*(y[t:t + 1] for y in x)) for t in range(N)])
    return o.cpu(), st.f32.cpu().view(HEADS, DV, DK)


@pytest.mark.parametrize("how,delta,diag", WALKED)
def test_a_negative_decay_multiplies(how, delta, diag):
    st, S = state(1, HEADS, DK, DV, delta, diag)
    q, k, v, alpha, beta = tokens(N, HEADS, 1, DK, DV, torch.float32, 80, diag)
    alpha[AT, 1] = -0.75
    alpha[AT + 3, 0] = -1.0
    want, end = recur(S[0], q, k, v, alpha, beta, delta)[:2]
    o, got = run(st, how, (q, k, v, alpha, beta))
    assert rel(o, want) <= 64 * U32 and rel(got, end) <= 64 * U32


@pytest.mark.parametrize("how,delta,diag", WALKED)
@pytest.mark.parametrize("tiny", [1e-39, 2.0 ** -126, 0.0])
def test_a_tiny_decay_multiplies(how, delta, diag, tiny):
    # nothing is written from the tiny decay on, so the state is fl(alpha S), subnormals kept
    st, _ = state(1, HEADS, DK, DV, delta, diag)
    x = tokens(N, HEADS, 1, DK, DV, torch.float32, 81, diag)
    _, before = run(st, how, x)
    alpha, beta = torch.ones_like(x[3]), torch.zeros_like(x[4])
    alpha[0] = tiny
    _, got = run(st, how, (*x[:3], alpha, beta))
    assert torch.equal(got, before * torch.tensor(tiny))
    assert tiny == 0.0 or bool((got != 0).any())


@pytest.mark.parametrize("how,delta,diag", WALKED)
def test_a_nan_decay_stays_in_its_head(how, delta, diag):
    st, _ = state(1, HEADS, DK, DV, delta, diag)
    start = st.f32.clone()
    x = list(tokens(N, HEADS, 1, DK, DV, torch.float32, 82, diag))
    o, S = run(st, how, x)
    x[3] = x[3].clone()
    x[3][AT, 1] = float("nan")
    st.f32.copy_(start)
    ob, Sb = run(st, how, x)
    assert bool(ob[AT:, 1].isnan().all()) and bool(Sb[1].isnan().all())
    assert torch.equal(ob[:AT], o[:AT]) and torch.equal(ob[:, ::2], o[:, ::2])
    assert torch.equal(Sb[::2], S[::2])
