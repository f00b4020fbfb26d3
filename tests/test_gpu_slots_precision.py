"""How far attend's chunk form may be off where an output's terms cancel (GPU).

The operands of a 16-bit output are sums of two bf16 parts, of an fp32 output three.  Two parts miss
at most 2^-16 of a value (half a step, 2^-8, of the first part's remainder, itself at most 2^-8), so
terms that cancel but for what two parts miss give 0 where the exact sum is up to 2^-16 B, B the
terms by their absolute values; binary16 inputs, of two parts themselves, add the products of second
parts, 3 * 2^-16 B in all.  fp32 sums add (3 T + Dk + 16) u B, u = 2^-24, for T tokens.
"""
import pytest
import torch

from tests.slots_ref import U32, batch_ref, half_step
from tests.test_gpu_slots import DEV, TYPES, state

pytestmark = pytest.mark.gpu
PARTS = {"bf16": 2.0 ** -16, "f16": 3 * 2.0 ** -16, "f32": 0.0}
DK = DV = 64


def two_parts(x):
    first = x.bfloat16().float()
    return first + (x - first).bfloat16().float()


def hard_value():
    """The fp32 number of many in [1, 2) that its two parts miss by most."""
    x = 1 + torch.rand(1 << 16, generator=torch.Generator().manual_seed(100))
    miss = (x - two_parts(x)).abs()
    assert 2.0 ** -18 < float(miss.max()) <= 2.0 ** -15      # 2^-16 of values up to 2
    return x[miss.argmax()]


def check(io, S, fresh, q, k, v, alpha, beta):
    dtype, n = TYPES[io], q.shape[0]
    st, _ = state(1, 1, DK, DV)
    st.f32.copy_(S.view(st.f32.shape))
    x = [y.to(dtype) for y in (q, k, v)] + [alpha, beta]
    o = st.attend(*(y.to(DEV) for y in x), torch.tensor([0, n], dtype=torch.int32, device=DEV),
                  fresh=torch.tensor([fresh], device=DEV)).double().cpu()
    want, _, B, _ = batch_ref(S, [0], [fresh], [0, n], *x)
    bound = half_step(dtype) * want.abs() + (PARTS[io] + (3 * n + DK + 16) * U32) * B
    if io == "f16":
        bound = bound + 2.0 ** -25
    assert float(((o - want).abs() - bound).max()) <= 0
    return o, want


@pytest.mark.parametrize("io", TYPES)
def test_a_state_whose_products_cancel(io):
    x = hard_value()
    S = torch.full((1, 1, DV, DK), float(x))
    S[..., 1::2] = two_parts(x)
    q = torch.ones(1, 1, DK)
    q[..., 1::2] = -1
    o, want = check(io, S, False, q, torch.zeros(1, 1, DK), torch.zeros(1, 1, DV), torch.ones(1, 1), torch.zeros(1, 1))
    assert bool((want != 0).all())
    if io == "f32":                              # the third part is there
        assert float((o / want - 1).abs().max()) < 0.1


@pytest.mark.parametrize("io", TYPES)
def test_tokens_whose_products_cancel(io):
    # two writes to the same key, taken back by the second but for what two parts miss
    x = hard_value()
    q = torch.zeros(2, 1, DK)
    q[..., 3] = 1
    v = torch.ones(2, 1, DV)
    v[1] = -1
    o, want = check(io, torch.zeros(1, 1, DV, DK), True, q, q.clone(), v, torch.ones(2, 1),
                    torch.stack([x, two_parts(x)])[:, None])
    assert bool((want[1] != 0).all())
    if io == "f32":
        assert float((o[1] / want[1] - 1).abs().max()) < 0.1
