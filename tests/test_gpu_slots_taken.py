"""Which entry of a call takes a slot: the first that has something to do with it (GPU)."""
import pytest
import torch

import quantized_recurrent_state_amd as lsq
from tests.slots_ref import batch_ref, tokens
from tests.test_gpu_slots import DEV, check_out, check_state, offsets, state

pytestmark = pytest.mark.gpu


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device=DEV)


def taken(lens, slots, n):
    """The slots with -1 in the place of an entry that is refused: a slot beyond n, or one that an
    earlier entry with tokens names."""
    out, seen = [], set()
    for length, s in zip(lens, slots):
        ok = 0 <= s < n and s not in seen
        out.append(s if ok else -1)
        if ok and length:
            seen.add(s)
    return out


@pytest.mark.parametrize("delta,diag", [(0, 0), (1, 0), (0, 1)])
@pytest.mark.parametrize("lens,slots", [([0, 20, 5], [2, 2, 1]), ([0, 0, 7, 0, 9], [1, 3, 3, 3, 1]),
                                        ([0, 6, 0, 6, 6], [0, 0, 0, 0, 1]),
                                        ([0, 1500, 0, 1300], [3, 3, 0, 0])], ids=str)
def test_an_empty_sequence_takes_no_slot(lens, slots, delta, diag):
    # 1500 and 1300 tokens of one head are cut into segments (scalar decay, delta 0)
    st, S = state(4, 1, 64, 64, delta, diag)
    n, cu = sum(lens), offsets(lens)
    x = tokens(n, 1, 1, 64, 64, torch.float32, 70, diag)
    o = st.attend(*(y.to(DEV) for y in x), i32(*cu), slots=i32(*slots))
    does = taken(lens, slots, 4)
    want, pool, ao, mag = batch_ref(S, does, None, cu, *x, delta)
    for i, s in enumerate(does):             # what is refused says so
        if s < 0:
            assert bool(o[cu[i]:cu[i + 1]].isnan().all())
    if delta:                                # signs mix in the correction: 2-norm only
        live = ~want.isnan()
        assert float((o.double().cpu() - want)[live].norm() / want[live].norm()) <= 64 * 2.0 ** -24
        assert float((st.f32.double().cpu().view(pool.shape) - pool).norm() / pool.norm()) <= 64 * 2.0 ** -24
    else:
        check_out(o, want, ao, max(lens), 64, torch.float32)
        check_state(st, pool, mag, max(lens))


@pytest.mark.parametrize("group", [32, 0])
def test_a_copy_without_a_source_takes_no_slot(group):
    f, _ = state(4, 2, 64, 64)
    cfg = lsq.LsqConfig(5, 2, 64, 64, 8, group, lsq.POLICY_DYNAMIC)
    cache = lsq.LsqState(cfg, device=DEV).zero()
    # pages 1 and 4 are first named with a padded source and one beyond the handle
    cache.store_slots(f, slots=i32(1, 4, 1, 4, 1, 0), src_slots=i32(-1, 9, 2, 3, 0, 4))
    whole = torch.zeros((5, 2 * 64, 64), device=DEV)
    whole[1], whole[4] = f.f32.view(4, 128, 64)[2], f.f32.view(4, 128, 64)[3]
    want = lsq.LsqState(cfg, device=DEV).zero().calibrate(whole.view(10, 64, 64))
    assert torch.equal(cache.codes, want.codes) and torch.equal(cache.scales, want.scales)
    back, _ = state(4, 2, 64, 64, seed=2)
    kept = back.f32.clone().view(4, -1)
    cache.load_slots(back, slots=i32(-3, 5, 1, 4, 4), dst_slots=i32(0, 3, 0, 3, 0))
    d = want.dequantize().view(5, -1)
    kept[0], kept[3] = d[1], d[4]
    assert torch.equal(back.f32.view(4, -1), kept)
