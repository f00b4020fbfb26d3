"""The slot operators on the GPU: prompts (attend), single tokens (step_slots), store and load.

Tolerances (fixed before the first run).  u = 2^-24.  With every term of the recurrence taken by
its absolute value (A for the state, B for the output) the kernels' fp32 sums are off by at most
n u A, n the roundings on the way: per token a decay, a gate and a write (3), the decays' own
logarithms and exponentials (8 u in all), and dk terms of a dot product for the output; the
output is then rounded once, half a step of its type.  Those are worst cases, a sum of many
independent roundings is far below them, so the whole state is also held to 16 u in the 2-norm,
and a 16-bit output to the half step itself.
"""
import pytest
import torch

import quantized_recurrent_state_amd as lsq
from tests.slots_ref import U32, batch_ref, half_step, rel, tokens

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def state(slots, heads, dk, dv, delta=0, diag=0, seed=1, scale=0.3):
    st = lsq.LsqState(lsq.LsqConfig(batch=slots, heads=heads, dk=dk, dv=dv, bits=32, group=1,
                                    policy=lsq.POLICY_NONE, delta=delta, decay=diag), device=DEV)
    g = torch.Generator().manual_seed(seed)
    S = torch.randn((slots, heads, dv, dk), generator=g) * scale
    st.f32.copy_(S.view(st.f32.shape))
    return st, S


def offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return cu


def check_out(o, want, mag, T, dk, dtype):
    """Every written element within half a step of its type plus the fp32 sums' bound."""
    o = o.double().cpu()
    live = ~want.isnan()
    assert o[live].isfinite().all()
    bound = half_step(dtype) * want.abs() + (3 * T + dk + 16) * U32 * mag * (1 + half_step(dtype))
    if dtype == torch.float16:
        bound = bound + 2.0 ** -25           # half a step of a subnormal
    over = ((o - want).abs() - bound)[live]
    assert float(over.max()) <= 0, f"off by {float(over.max())} over the bound"


def check_state(st, pool, mag, T):
    S = st.f32.double().cpu().view(pool.shape)
    over = (S - pool).abs() - (3 * T + 8) * U32 * mag
    assert float(over.max()) <= 0
    assert rel(S, pool) <= 16 * U32


def run_attend(lens, heads, qk_heads, dk, dv, dtype, slots=None, fresh=None, n_slots=None, pad=0,
               slow=False, delta=0, diag=0, tail=0, seed=3, o_pad=0, alpha0=()):
    cu = offsets(lens)
    n = cu[-1] + tail
    slots = list(range(len(lens))) if slots is None else slots
    n_slots = n_slots or max(slots + [0]) + 2
    st, S = state(n_slots, heads, dk, dv, delta, diag)
    q, k, v, alpha, beta = tokens(n, heads, qk_heads, dk, dv, dtype, seed, diag, slow, pad)
    for t in alpha0:
        alpha[t] = 0.0

    def dev(x):
        """x on the device with its own strides."""
        if pad and x.dim() == 3 and x.dtype == dtype and x.shape[0]:
            base = x.as_strided((x.shape[0], x.stride(0)), (x.stride(0), 1))
            return base.to(DEV)[:, :x.shape[1] * x.shape[2]].unflatten(1, x.shape[1:])
        return x.to(DEV)

    wide = torch.full((n, heads * dv + o_pad), float("nan"), dtype=dtype, device=DEV)
    o = wide[:, :heads * dv].unflatten(1, (heads, dv))
    f = None if fresh is None else torch.tensor(fresh, device=DEV)
    got = st.attend(dev(q), dev(k), dev(v), dev(alpha), dev(beta),
                    torch.tensor(cu, dtype=torch.int32, device=DEV),
                    slots=torch.tensor(slots, dtype=torch.int32, device=DEV), fresh=f, o=o)
    assert got is o
    want, pool, ao, mag = batch_ref(S, slots, fresh, cu, q, k, v, alpha, beta, delta)
    T = max(lens)
    assert bool(o.cpu()[want.isnan()].isnan().all()), "a row that no sequence owns was written"
    if o_pad:
        assert bool(wide[:, heads * dv:].isnan().all())
    if delta:                                # the rank-one correction mixes signs: 2-norm only
        live = ~want.isnan()
        lim = half_step(dtype) + 64 * U32
        assert rel(o.cpu()[live], want[live]) <= lim
        assert rel(st.f32.cpu().view(pool.shape), pool) <= 64 * U32
    else:
        check_out(o, want, ao, T, dk, dtype)
        check_state(st, pool, mag, T)
        live = ~want.isnan()
        if live.any():
            assert rel(o.cpu()[live], want[live]) <= half_step(dtype) + 16 * U32
    return st


SHAPES = [(4, 4, 64, 64), (4, 2, 128, 128), (2, 1, 128, 64), (3, 3, 64, 80), (2, 2, 128, 200),
          (1, 1, 64, 16), (2, 1, 64, 7), (1, 1, 128, 1), (4, 1, 128, 130)]


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "x".join(map(str, s)))
def test_attend_shapes(io, shape):
    run_attend([70, 1, 33], *shape, TYPES[io], slots=[2, 0, 3], fresh=[False, True, False])


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 300])
def test_attend_lengths(io, n):
    run_attend([n], 2, 1, 64, 64, TYPES[io])
    run_attend([n], 1, 1, 128, 128, TYPES[io], fresh=[True])


@pytest.mark.parametrize("io", TYPES)
def test_attend_empty_padded_and_outside(io):
    # empty sequences, a padded entry whose rows stay, tokens behind the last sequence
    st = run_attend([0, 40, 0, 17, 5], 2, 2, 64, 64, TYPES[io], slots=[4, 1, 0, -1, 6],
                    fresh=[True, False, False, True, False], tail=9)
    assert bool(st.f32.isfinite().all())


@pytest.mark.parametrize("io", TYPES)
def test_attend_strided_rows(io):
    # q, k, v as slices of a wider projection, o inside a wider row
    run_attend([66, 20], 2, 2, 64, 64, TYPES[io], pad=16, o_pad=8)
    run_attend([40, 9], 2, 1, 128, 72, TYPES[io], pad=8, o_pad=3)


@pytest.mark.parametrize("io", TYPES)
def test_attend_slow_decay_and_resets(io):
    run_attend([400], 1, 1, 64, 64, TYPES[io], slow=True)
    # alpha = 0 forgets: at the first token, inside a chunk, at a chunk's border, two in a row
    run_attend([150], 2, 2, 64, 64, TYPES[io], alpha0=(0, 20, 21, 64, 128))


def test_attend_fast_decay():
    # decays so strong that a chunk's product leaves the range of fp32
    lens = [130]
    st, S = state(2, 2, 64, 64)
    q, k, v, alpha, beta = tokens(130, 2, 2, 64, 64, torch.float32, 4)
    alpha = alpha ** 40
    o = st.attend(*(x.to(DEV) for x in (q, k, v, alpha, beta)),
                  torch.tensor([0, 130], dtype=torch.int32, device=DEV))
    want, pool, ao, mag = batch_ref(S, [0], None, offsets(lens), q, k, v, alpha, beta)
    check_out(o, want, ao, 130, 64, torch.float32)
    check_state(st, pool, mag, 130)


@pytest.mark.parametrize("io", ["bf16", "f32"])
def test_attend_many_sequences(io):
    lens = [(7 * i) % 23 for i in range(150)]
    slots = [(11 * i) % 160 for i in range(150)]
    run_attend(lens, 1, 1, 64, 64, TYPES[io], slots=slots, n_slots=160)


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", [(1, 0), (0, 1), (1, 1)])
def test_attend_delta_and_diagonal(io, delta, diag):
    run_attend([40, 1, 66], 2, 1, 128, 72, TYPES[io], delta=delta, diag=diag, fresh=[False, True, False])
    run_attend([9], 2, 2, 64, 64, TYPES[io], delta=delta, diag=diag)


def test_attend_fresh_ignores_a_spoilt_slot():
    st, S = state(3, 2, 64, 64)
    st.f32.fill_(float("nan"))
    q, k, v, alpha, beta = tokens(70, 2, 2, 64, 64, torch.bfloat16, 5)
    o = st.attend(*(x.to(DEV) for x in (q, k, v, alpha, beta)),
                  torch.tensor([0, 70], dtype=torch.int32, device=DEV),
                  slots=torch.tensor([1], dtype=torch.int32, device=DEV),
                  fresh=torch.tensor([True], device=DEV))
    want, pool, ao, _ = batch_ref(S, [1], [True], [0, 70], q, k, v, alpha, beta)
    check_out(o, want, ao, 70, 64, torch.bfloat16)
    got = st.f32.view(3, 2, 64, 64).cpu()
    assert rel(got[1], pool[1]) <= 16 * U32
    assert bool(got[0].isnan().all()) and bool(got[2].isnan().all())


def test_refused_slots_touch_no_state_and_say_so():
    # one slot twice and one beyond the handle: the first of the two is carried out
    st, S = state(4, 2, 64, 64)
    n = 3 * 20
    q, k, v, alpha, beta = tokens(n, 2, 2, 64, 64, torch.bfloat16, 6)
    cu = torch.tensor([0, 20, 40, 60], dtype=torch.int32, device=DEV)
    o = st.attend(*(x.to(DEV) for x in (q, k, v, alpha, beta)), cu,
                  slots=torch.tensor([2, 2, 4], dtype=torch.int32, device=DEV))
    want, pool, ao, mag = batch_ref(S, [2], None, [0, 20], q, k, v, alpha, beta)
    check_out(o[:20], want[:20], ao[:20], 20, 64, torch.bfloat16)
    check_state(st, pool, mag, 20)
    assert bool(o[20:].isnan().all())
    st, S = state(4, 2, 64, 64)
    o = st.step_slots(*(x[:3].to(DEV) for x in (q, k, v, alpha, beta)),
                      slots=torch.tensor([3, 9, 3], dtype=torch.int32, device=DEV))
    want, pool, ao, mag = batch_ref(S, [3], None, [0, 1], q, k, v, alpha, beta)
    check_out(o[:1], want[:1], ao[:1], 1, 64, torch.bfloat16)
    check_state(st, pool, mag, 1)
    assert bool(o[1:].isnan().all())


def test_spoilt_offsets_stay_inside():
    # decreasing, negative and too large offsets: clamped, no row outside is touched
    st, S = state(4, 1, 64, 64)
    q, k, v, alpha, beta = tokens(30, 1, 1, 64, 64, torch.float32, 7)
    cu = torch.tensor([-5, 10, 4, 1 << 30], dtype=torch.int32, device=DEV)
    o = st.attend(*(x.to(DEV) for x in (q, k, v, alpha, beta)), cu)
    assert bool(o[10:].isfinite().all()) and bool(st.f32.isfinite().all())
    assert torch.equal(st.f32.view(4, 1, 64, 64)[1].cpu(), S[1])


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", [(0, 0), (1, 0), (0, 1), (1, 1)])
@pytest.mark.parametrize("shape", [(4, 2, 128, 128), (3, 3, 64, 80), (2, 1, 128, 7), (1, 1, 64, 200)],
                         ids=lambda s: "x".join(map(str, s)))
def test_step_slots(io, delta, diag, shape):
    heads, hk, dk, dv = shape
    dtype = TYPES[io]
    slots, fresh = [5, -1, 0, 2], [False, False, True, False]
    st, S = state(6, heads, dk, dv, delta, diag)
    q, k, v, alpha, beta = tokens(4, heads, hk, dk, dv, dtype, 8, diag)
    o = torch.full((4, heads, dv), float("nan"), dtype=dtype, device=DEV)
    st.step_slots(*(x.to(DEV) for x in (q, k, v, alpha, beta)),
                  slots=torch.tensor(slots, dtype=torch.int32, device=DEV),
                  fresh=torch.tensor(fresh, device=DEV), o=o)
    want, pool, ao, mag = batch_ref(S, slots, fresh, [0, 1, 2, 3, 4], q, k, v, alpha, beta, delta)
    assert bool(o[1].isnan().all())
    live = ~want.isnan()
    if delta:
        assert rel(o.cpu()[live], want[live]) <= half_step(dtype) + 64 * U32
        assert rel(st.f32.cpu().view(pool.shape), pool) <= 64 * U32
    else:
        check_out(o, want, ao, 1, dk, dtype)
        check_state(st, pool, mag, 1)


def test_step_slots_equals_the_fp32_step():
    # the same arithmetic as the handle's own step: equal states, outputs equal up to the sum's order
    for delta in (0, 1):
        st, S = state(6, 4, 128, 128, delta)
        ref, _ = state(6, 4, 128, 128, delta)
        q, k, v, alpha, beta = tokens(6, 4, 4, 128, 128, torch.float32, 9)
        args = [x.to(DEV) for x in (q, k, v, alpha, beta)]
        o = st.step_slots(*args)
        w = ref.step(*(x.flatten(0, 1).contiguous() for x in args))
        assert rel(o.cpu().flatten(0, 1), w.double().cpu()) <= 16 * U32
        assert rel(st.f32.cpu(), ref.f32.double().cpu()) <= (16 * U32 if delta else 0)


STORE = [(b, g, f, p) for b in (4, 8) for g in (16, 32, 64, 128, 0) for f in (0, 1, 2)
         for p in (lsq.POLICY_DYNAMIC, lsq.POLICY_PERSISTENT, lsq.POLICY_YOKED)
         if (g or (f == 0 and p != lsq.POLICY_YOKED)) and (f == 0 or p == lsq.POLICY_DYNAMIC)]


@pytest.mark.parametrize("bits,group,fmt,policy", STORE)
@pytest.mark.parametrize("dk,dv", [(128, 128), (64, 80), (128, 3)])
def test_store_and_load_are_calibrate_and_dequantize(bits, group, fmt, policy, dk, dv):
    """Bit for bit the whole handle's calibration and read-back, slot by slot."""
    if group > dk:
        pytest.skip("a group is at most a row")
    heads, pages = 3, 7
    f, S = state(5, heads, dk, dv)
    f.f32[:dv].mul_(0.0)                     # a head of zeros: scale 0
    cfg = lsq.LsqConfig(batch=pages, heads=heads, dk=dk, dv=dv, bits=bits, group=group, policy=policy,
                        scale_fmt=fmt)
    cache = lsq.LsqState(cfg, device=DEV).zero()
    src, dst = [4, 0, 0, 2, 1], [6, 0, 3, -1, 2]
    cache.store_slots(f, slots=torch.tensor(dst, dtype=torch.int32, device=DEV),
                      src_slots=torch.tensor(src, dtype=torch.int32, device=DEV))
    want = lsq.LsqState(cfg, device=DEV).zero()
    whole = torch.zeros((pages, heads * dv, dk), device=DEV)
    for s, d in zip(src, dst):
        if d >= 0:
            whole[d] = f.f32.view(5, heads * dv, dk)[s]
    want.calibrate(whole.view(pages * heads, dv, dk))
    assert torch.equal(cache.codes, want.codes)
    assert torch.equal(cache.scales.float(), want.scales.float())
    if policy == lsq.POLICY_YOKED:
        assert torch.equal(cache.ref, want.ref)
    back, _ = state(8, heads, dk, dv, seed=2)
    before = back.f32.clone().view(8, -1)
    to = [7, 1, 0]
    cache.load_slots(back, slots=torch.tensor([6, 0, 2], dtype=torch.int32, device=DEV),
                     dst_slots=torch.tensor(to, dtype=torch.int32, device=DEV))
    d = want.dequantize().view(pages, -1)
    before[to] = d[[6, 0, 2]]
    assert torch.equal(back.f32.view(8, -1), before)


def test_store_and_load_refuse_on_the_device():
    f, S = state(4, 2, 64, 64)
    cache = lsq.LsqState(lsq.LsqConfig(3, 2, 64, 64, 8, 64, lsq.POLICY_DYNAMIC), device=DEV).zero()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    # a page twice (the first counts), a page and a source beyond the handles, padded ones
    cache.store_slots(f, slots=i32(1, 1, 3, 0, -1, 2), src_slots=i32(2, 3, 0, 4, 1, -7))
    want = lsq.LsqState(cache.cfg, device=DEV).zero()
    whole = torch.zeros((3, 2 * 64, 64), device=DEV)
    whole[1] = f.f32.view(4, 128, 64)[2]
    want.calibrate(whole.view(6, 64, 64))
    assert torch.equal(cache.codes, want.codes) and torch.equal(cache.scales, want.scales)
    before = f.f32.clone()
    cache.load_slots(f, slots=i32(3, 1, -1), dst_slots=i32(0, 5, 1))
    assert torch.equal(f.f32, before)


def test_prompt_cache_fork_and_decode():
    """A run as a serving program makes it: a prompt, its state put into the cache, two requests
    forked from it, a second piece of prompt and then tokens for both, then decoding on the
    quantised state itself."""
    heads, dk, dv, dtype = 4, 128, 128, torch.bfloat16
    st, _ = state(6, heads, dk, dv)
    cache = lsq.LsqState(lsq.LsqConfig(4, heads, dk, dv, 8, 64, lsq.POLICY_DYNAMIC), device=DEV).zero()
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device=DEV)
    q, k, v, alpha, beta = tokens(100 + 30 + 17 + 6, heads, 2, dk, dv, dtype, 10)
    d = [x.to(DEV) for x in (q, k, v, alpha, beta)]
    st.attend(*(x[:100] for x in d), i32(0, 100), slots=i32(3), fresh=torch.tensor([True], device=DEV))
    cache.store_slots(st, slots=i32(2), src_slots=i32(3))
    cache.load_slots(st, slots=i32(2, 2), dst_slots=i32(0, 5))
    _, S1, _, _ = batch_ref(torch.zeros(1, heads, dv, dk), [0], None, [0, 100], *(x[:100] for x in (q, k, v, alpha, beta)))[0:4]
    base = cache.dequantize().view(4, heads, dv, dk)[2].cpu()
    # what the cache holds is the prompt's state within half an INT8 step of each group's largest
    step = S1[0].view(heads, dv, 2, 64).abs().amax(-1, keepdim=True) / 127
    err = (base.double() - S1[0]).view(heads, dv, 2, 64).abs()
    assert bool((err <= step * (0.5 + 130 * U32 * 127)).all())
    piece = [x[100:147] for x in (q, k, v, alpha, beta)]
    o = st.attend(*(x.to(DEV) for x in piece), i32(0, 30, 47), slots=i32(5, 0))
    pool = torch.zeros(6, heads, dv, dk)
    pool[0] = pool[5] = base
    want, pool, ao, mag = batch_ref(pool, [5, 0], None, [0, 30, 47], *piece)
    check_out(o, want, ao, 30, dk, dtype)
    for t in range(3):
        tok = [x[147 + 2 * t:149 + 2 * t] for x in (q, k, v, alpha, beta)]
        o = st.step_slots(*(x.to(DEV) for x in tok), slots=i32(0, 5))
        want, pool, ao, mag = batch_ref(pool, [0, 5], None, [0, 1, 2], *tok)
        check_out(o, want, ao, 40, dk, dtype)
    cache.store_slots(st, slots=i32(0, 1), src_slots=i32(5, 0))
    one = [x[:4].float().to(DEV) for x in (q, k, v, alpha, beta)]
    o = cache.step(*(x.repeat_interleave(2, 1).flatten(0, 1).contiguous() if x.dim() == 3 and x.shape[1] == 2
                     else x.flatten(0, 1).contiguous() for x in one))
    assert bool(o.isfinite().all())


def test_other_stream_and_graph_replays():
    """The calls on a stream of their own, then captured: every replay equals the eager run, with
    other slots read at replay."""
    heads, dk, dv, dtype = 4, 128, 128, torch.bfloat16
    q, k, v, alpha, beta = (x.to(DEV) for x in tokens(700, heads, 2, dk, dv, dtype, 11))
    cu = torch.tensor([0, 600, 630, 700], dtype=torch.int32, device=DEV)
    one = [x[:3].contiguous() for x in (q, k, v, alpha, beta)]
    cfg = lsq.LsqConfig(6, heads, dk, dv, 4, 32, lsq.POLICY_DYNAMIC)

    def program(st, cache, slots, pages, stream=None):
        o = st.attend(q, k, v, alpha, beta, cu, slots=slots, stream=stream)
        cache.store_slots(st, slots=pages, src_slots=slots, stream=stream)
        cache.load_slots(st, slots=pages, dst_slots=slots, stream=stream)
        return o, st.step_slots(*one, slots=slots, stream=stream)

    def i32(*x):
        return torch.tensor(x, dtype=torch.int32, device=DEV)

    def eager(slots, pages, stream=None):
        st, _ = state(6, heads, dk, dv)
        cache = lsq.LsqState(cfg, device=DEV).zero()
        torch.cuda.synchronize()
        o, p = program(st, cache, i32(*slots), i32(*pages), stream)
        torch.cuda.synchronize()
        return o, p, st.f32, cache.codes

    a, b = eager((4, 0, 2), (1, 5, 3)), eager((1, 5, 3), (0, 2, 4))
    for x, y in zip(a, eager((4, 0, 2), (1, 5, 3), torch.cuda.Stream())):
        assert torch.equal(x, y)
    st, S = state(6, heads, dk, dv)
    S = S.to(DEV).view(st.f32.shape)
    cache = lsq.LsqState(cfg, device=DEV).zero()
    slots, pages = i32(4, 0, 2), i32(1, 5, 3)
    program(st, cache, slots, pages)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o, p = program(st, cache, slots, pages)
    for want, s, g in ((a, (4, 0, 2), (1, 5, 3)), (b, (1, 5, 3), (0, 2, 4)), (a, (4, 0, 2), (1, 5, 3))):
        st.f32.copy_(S)
        cache.zero()
        slots.copy_(i32(*s))
        pages.copy_(i32(*g))
        graph.replay()
        torch.cuda.synchronize()
        for x, y in zip((o, p, st.f32, cache.codes), want):
            assert torch.equal(x, y)


def test_attend_repeats_bit_for_bit():
    first = None
    for _ in range(2):
        st, _ = state(2, 2, 128, 128)
        q, k, v, alpha, beta = (x.to(DEV) for x in tokens(2000, 2, 2, 128, 128, torch.bfloat16, 12))
        o = st.attend(q, k, v, alpha, beta, torch.tensor([0, 1900, 2000], dtype=torch.int32, device=DEV))
        if first is None:
            first = o, st.f32.clone()
        else:
            assert torch.equal(o, first[0]) and torch.equal(st.f32, first[1])


@pytest.mark.parametrize("io", TYPES)
def test_attend_long_and_segments(io):
    # long enough to be taken in segments, beside short sequences
    run_attend([1500, 3, 700, 64], 1, 1, 64, 64, TYPES[io], slots=[1, 0, 3, 2],
               fresh=[False, False, True, False], seed=13)
    run_attend([2100], 1, 1, 128, 128, TYPES[io], seed=14, slow=True)


@pytest.mark.parametrize("io", ["bf16", "f32"])
@pytest.mark.parametrize("seqs", [9, 70])
def test_attend_cuts_only_the_long_ones(io, seqs):
    """Few long sequences among many short ones: the long ones are cut, wherever they stand."""
    lens = [(5 * i) % 37 for i in range(seqs)]
    lens[2], lens[seqs - 3] = 1700, 2600
    run_attend(lens, 1, 1, 64, 64, TYPES[io], slots=[(7 * i) % (seqs + 4) for i in range(seqs)] if seqs != 70
               else [(7 * i) % 73 for i in range(seqs)], n_slots=seqs + 4, fresh=[i % 3 == 0 for i in range(seqs)],
               seed=15)


def test_attend_refuses_and_pads_cut_sequences():
    st, S = state(4, 1, 64, 64)
    q, k, v, alpha, beta = tokens(4 * 1500, 1, 1, 64, 64, torch.bfloat16, 16)
    o = torch.full((6000, 1, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    cu = torch.tensor([0, 1500, 3000, 4500, 6000], dtype=torch.int32, device=DEV)
    st.attend(*(x.to(DEV) for x in (q, k, v, alpha, beta)), cu,
              slots=torch.tensor([3, -1, 3, 8], dtype=torch.int32, device=DEV), o=o)
    want, pool, ao, mag = batch_ref(S, [3], None, [0, 1500], q, k, v, alpha, beta)
    check_out(o[:1500], want[:1500], ao[:1500], 1500, 64, torch.bfloat16)
    check_state(st, pool, mag, 1500)
    assert bool((o[1500:3000] == 7).all()) and bool(o[3000:].isnan().all())


def test_spoilt_offsets_of_long_sequences_stay_inside():
    # the same tokens named twice: no slot but the named ones, no memory outside, is touched
    st, S = state(6, 1, 64, 64)
    q, k, v, alpha, beta = (x.to(DEV) for x in tokens(6000, 1, 1, 64, 64, torch.bfloat16, 17))
    guard = torch.full((6002, 1, 64), 5.0, dtype=torch.bfloat16, device=DEV)
    cu = torch.tensor([0, 6000, 0, 6000, 0, 6000], dtype=torch.int32, device=DEV)
    st.attend(q, k, v, alpha, beta, cu, slots=torch.tensor([0, 1, 2, 3, 4], dtype=torch.int32, device=DEV),
              o=guard[1:6001])
    assert bool((guard[0] == 5).all()) and bool((guard[6001] == 5).all())
    assert torch.equal(st.f32.view(6, 1, 64, 64)[5].cpu(), S[5])


@pytest.mark.parametrize("io", TYPES)
def test_attend_broadcast_inputs(io):
    # one q, k or v row shared by all tokens (stride 0), with a last chunk that is not full
    dtype, n, heads, dk, dv = TYPES[io], 75, 2, 64, 64
    st, S = state(1, heads, dk, dv)
    q, k, v, alpha, beta = tokens(n, heads, heads, dk, dv, dtype, 18)
    q, k, v = (x[:1].expand(n, heads, 64) for x in (q, k, v))
    dev = [x[:1].to(DEV).expand(n, heads, 64) for x in (q, k, v)]
    o = st.attend(*dev, alpha.to(DEV), beta.to(DEV), torch.tensor([0, n], dtype=torch.int32, device=DEV))
    want, pool, ao, mag = batch_ref(S, [0], None, [0, n], q, k, v, alpha, beta)
    check_out(o, want, ao, n, dk, dtype)
    check_state(st, pool, mag, n)
    o = st.step_slots(*(x[:1] for x in dev), alpha[:1].to(DEV), beta[:1].to(DEV))
    want, pool, ao, mag = batch_ref(pool, [0], None, [0, 1], q, k, v, alpha, beta)
    check_out(o, want[:1], ao[:1], n + 1, dk, dtype)


def test_attend_skips_rows_before_and_behind():
    # NaN in rows that no sequence owns reaches nothing
    st, S = state(2, 2, 64, 64)
    q, k, v, alpha, beta = tokens(120, 2, 2, 64, 64, torch.bfloat16, 19)
    for x in (q, k, v, alpha, beta):
        x[:11] = float("nan")
        x[61:64] = float("nan")
        x[110:] = float("nan")
    cu, slots = [11, 61, 64, 110], [0, -1, 1]
    o = st.attend(*(x.to(DEV) for x in (q, k, v, alpha, beta)), torch.tensor(cu, dtype=torch.int32, device=DEV),
                  slots=torch.tensor(slots, dtype=torch.int32, device=DEV),
                  o=torch.full((120, 2, 64), float("nan"), dtype=torch.bfloat16, device=DEV))
    want, pool, ao, mag = batch_ref(S, slots, None, cu, q, k, v, alpha, beta)
    assert bool(o.cpu()[want.isnan()].isnan().all())
    check_out(o, want, ao, 50, 64, torch.bfloat16)
    check_state(st, pool, mag, 50)


@pytest.mark.parametrize("io", TYPES)
def test_nothing_written_leaves_the_state_bit_for_bit(io):
    st, S = state(2, 2, 128, 128)
    q, k, v, alpha, beta = tokens(1700, 2, 2, 128, 128, TYPES[io], 20)
    alpha, beta = torch.ones_like(alpha), torch.zeros_like(beta)
    st.attend(*(x.to(DEV) for x in (q, k, v, alpha, beta)), torch.tensor([0, 1600, 1700], dtype=torch.int32, device=DEV))
    assert torch.equal(st.f32.cpu().view(S.shape), S)


def test_pools_and_strides_beyond_32_bits():
    """The last slots of a pool of more than 4 GiB, and rows more than 4 GiB apart."""
    heads, dk, dv, dtype = 32, 128, 128, torch.bfloat16
    n_slots = 2200                               # 2 MiB each
    st = lsq.LsqState(lsq.LsqConfig(n_slots, heads, dk, dv, 32, 1, lsq.POLICY_NONE), device=DEV)
    st.f32.zero_()
    last = torch.randn((2, heads, dv, dk), generator=torch.Generator().manual_seed(21))
    st.f32.view(n_slots, heads, dv, dk)[-2:] = last.to(DEV)
    slots = torch.tensor([n_slots - 1, n_slots - 2], dtype=torch.int32, device=DEV)
    cache = lsq.LsqState(lsq.LsqConfig(n_slots, heads, dk, dv, 8, 64, lsq.POLICY_DYNAMIC), device=DEV)
    cache.store_slots(st, slots=slots, src_slots=slots)
    want = lsq.LsqState(lsq.LsqConfig(2, heads, dk, dv, 8, 64, lsq.POLICY_DYNAMIC), device=DEV)
    want.calibrate(last.view(-1, dv, dk).to(DEV))
    assert torch.equal(cache.codes.view(n_slots, -1)[-2:], want.codes.view(2, -1))
    cache.load_slots(st, slots=slots, dst_slots=slots)
    base = want.dequantize().view(2, heads, dv, dk).cpu()
    assert torch.equal(st.f32.view(n_slots, heads, dv, dk)[-2:].cpu(), base)
    assert not bool(st.f32.view(n_slots, -1)[0].any())
    # q and v as slices of rows of 8 MiB elements: token 300 lies 4.7 GiB behind token 0
    n, row = 300, 8 << 20
    q, k, v, alpha, beta = tokens(n, heads, 1, dk, dv, dtype, 22)
    wide = torch.zeros((n, row), dtype=dtype, device=DEV)
    wide[:, :dk] = q[:, 0].to(DEV)
    wide[:, 1024:1024 + heads * dv] = v.flatten(1).to(DEV)
    a, b = alpha.to(DEV), beta.to(DEV)
    cu = torch.tensor([0, n - 1], dtype=torch.int32, device=DEV)
    args = [wide[:, :dk].unflatten(1, (1, dk)), k.to(DEV), wide[:, 1024:1024 + heads * dv].unflatten(1, (heads, dv))]
    o = st.attend(*args, a, b, cu, slots=slots[:1])
    ref, pool, ao, mag = batch_ref(base[1:], [0], None, [0, n - 1], q, k, v, alpha, beta)
    check_out(o[:n - 1], ref[:n - 1], ao[:n - 1], n, dk, dtype)
    got = st.f32.view(n_slots, heads, dv, dk)[-1:].cpu()
    assert rel(got, pool) <= 16 * U32
    o = st.step_slots(*(x[n - 1:] for x in args), a[n - 1:], b[n - 1:], slots=slots[1:])
    ref, pool, ao, mag = batch_ref(base[:1], [0], None, [0, 1], *(x[n - 1:] for x in (q, k, v, alpha, beta)))
    check_out(o, ref, ao, 1, dk, dtype)
    assert rel(st.f32.view(n_slots, heads, dv, dk)[-2:-1].cpu(), pool) <= 16 * U32


def test_two_streams_and_two_graphs_with_cut_sequences():
    """Two batches on two streams at once, then two captured graphs replayed in turn: each has a
    workspace of its own, and every replay equals the eager run."""
    heads, dk, dv, dtype = 2, 64, 64, torch.bfloat16
    data = [[x.to(DEV) for x in tokens(3000, heads, heads, dk, dv, dtype, 23 + i)] for i in range(2)]
    cu = torch.tensor([0, 1400, 3000], dtype=torch.int32, device=DEV)
    slots = [torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 1], [3, 2])]

    def eager(i):
        st, _ = state(4, heads, dk, dv)
        return st.attend(*data[i], cu, slots=slots[i]), st.f32.view(4, -1)[slots[i].long()]

    want = [eager(0), eager(1)]
    st, S = state(4, heads, dk, dv)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    got = [st.attend(*data[i], cu, slots=slots[i], stream=streams[i]) for i in range(2)]
    torch.cuda.synchronize()
    for i in range(2):
        assert torch.equal(got[i], want[i][0])
        assert torch.equal(st.f32.view(4, -1)[slots[i].long()], want[i][1])
    S = S.to(DEV).view(st.f32.shape)
    graphs, outs = [], []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(st.attend(*data[i], cu, slots=slots[i]))
        graphs.append(g)
    for _ in range(3):
        st.f32.copy_(S)
        for i in (1, 0):
            graphs[i].replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[i][0])
            assert torch.equal(st.f32.view(4, -1)[slots[i].long()], want[i][1])


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")], ids=str)
@pytest.mark.parametrize("n,at", [(40, 5), (70, 31), (70, 32), (100, 95), (1500, 700)])
def test_a_value_that_is_not_finite_reaches_no_earlier_token(io, bad, n, at):
    # one element of v or k of one token: the outputs before it, and of v the other columns, keep
    # their bits; from it on the column (of k, the heads that share it) is not finite.  1500 tokens
    # of one head are cut into segments.
    heads = 2 if n < 1000 else 1
    st, _ = state(1, heads, 64, 80)
    start = st.f32.clone()
    q, k, v, alpha, beta = (x.to(DEV) for x in tokens(n, heads, 1, 64, 80, TYPES[io], 40))
    cu = torch.tensor([0, n], dtype=torch.int32, device=DEV)

    def run(k, v):
        st.f32.copy_(start)
        return st.attend(q, k, v, alpha, beta, cu), st.f32.clone().view(heads, 80, 64)

    o, S = run(k, v)
    assert bool(o.isfinite().all())
    for col in (0, 21, 79):
        vb = v.clone()
        vb[at, heads - 1, col] = bad
        ob, Sb = run(k, vb)
        assert torch.equal(ob[:at], o[:at])
        assert not bool(ob[at:, heads - 1, col].isfinite().any())
        assert not bool(Sb[heads - 1, col].isfinite().any())
        ob[at:, heads - 1, col] = o[at:, heads - 1, col]
        Sb[heads - 1, col] = S[heads - 1, col]
        assert torch.equal(ob, o) and torch.equal(Sb, S)
    kb = k.clone()
    kb[at, 0, 17] = bad
    ob, Sb = run(kb, v)
    assert torch.equal(ob[:at], o[:at])
    assert not bool(ob[at:].isfinite().any())
    assert torch.equal(Sb[..., :17], S[..., :17]) and torch.equal(Sb[..., 18:], S[..., 18:])


@pytest.mark.parametrize("io", TYPES)
@pytest.mark.parametrize("delta,diag", [(1, 0), (0, 1), (1, 1)])
def test_a_walked_prompt_equals_its_single_tokens(io, delta, diag):
    # prompts that walk (few of them and many) and the recurrent form: the same bits
    for seqs, n in ((1, 1), (1, 2), (2, 5), (9, 4)):
        heads, dk, dv = 32, 64, 40
        st, _ = state(seqs, heads, dk, dv, delta, diag)
        start = st.f32.clone()
        x = [y.to(DEV) for y in tokens(seqs * n, heads, 4, dk, dv, TYPES[io], 50 + n, diag)]
        cu = torch.arange(0, seqs * n + 1, n, dtype=torch.int32, device=DEV)
        o = st.attend(*x, cu)
        S = st.f32.clone()
        st.f32.copy_(start)
        for t in range(n):
            one = st.step_slots(*(y[t::n].contiguous() for y in x))
            assert torch.equal(one, o[t::n])
        assert torch.equal(st.f32, S)


@pytest.mark.parametrize("io,e", [("f32", -90), ("f32", 100), ("bf16", -90), ("bf16", 100)])
def test_small_and_large_magnitudes_keep_the_accuracy(io, e):
    # v and the state scaled by a power of two: the outputs and the state scale with them.  Each side
    # is within 16 u of the definition in the 2-norm (outputs: and half a step of their type).
    st, _ = state(1, 2, 64, 80)
    start = st.f32.clone()
    q, k, v, alpha, beta = (x.to(DEV) for x in tokens(150, 2, 1, 64, 80, TYPES[io], 60))
    cu = torch.tensor([0, 150], dtype=torch.int32, device=DEV)
    o = st.attend(q, k, v, alpha, beta, cu).double()
    S = st.f32.double()
    st.f32.copy_(start * 2.0 ** e)
    oe = st.attend(q, k, v * 2.0 ** e, alpha, beta, cu).double() * 2.0 ** -e
    assert rel(st.f32.double().cpu() * 2.0 ** -e, S.cpu()) <= 32 * U32
    assert rel(oe.cpu(), o.cpu()) <= 2 * half_step(TYPES[io]) + 32 * U32


def test_a_negative_or_nan_alpha_gives_nan_from_its_token_on():
    st, _ = state(1, 3, 64, 64)
    start = st.f32.clone()
    q, k, v, alpha, beta = (x.to(DEV) for x in tokens(90, 3, 1, 64, 64, torch.bfloat16, 61))
    cu = torch.tensor([0, 90], dtype=torch.int32, device=DEV)
    o = st.attend(q, k, v, alpha, beta, cu)
    for bad in (-0.5, float("nan")):
        a = alpha.clone()
        a[45, 1] = bad
        st.f32.copy_(start)
        ob = st.attend(q, k, v, a, beta, cu)
        assert torch.equal(ob[:45], o[:45]) and torch.equal(ob[:, ::2], o[:, ::2])
        assert bool(ob[45:, 1].isnan().all()) and bool(st.f32.view(3, -1)[1].isnan().all())
    a = alpha.clone()
    outs = []
    for tiny in (0.0, 1e-39):                # both forget what was before
        a[45, 1] = tiny
        st.f32.copy_(start)
        outs.append((st.attend(q, k, v, a, beta, cu), st.f32.clone()))
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])
