"""Refusals of the slot calls (no GPU needed, no kernel launched).

The device pointers are never dereferenced: every call fails its checks, or has nothing to do,
before any launch.
"""
import ctypes

import pytest
import torch

import quantized_recurrent_state_amd as lsq
from quantized_recurrent_state_amd import _lib, slots

FAKE = 0x7F0000000000


def handle(**kw):
    base = dict(batch=4, heads=4, dk=128, dv=64, bits=32, group=1, policy=lsq.POLICY_NONE)
    base.update(kw)
    cfg = lsq.LsqConfig(**base)
    need = lsq.lsq_state_sizes(cfg)
    bufs = _lib.lsq_buffers(*(x for n in need for x in (FAKE if n else None, n)))
    h = ctypes.c_void_p()
    assert _lib.load().lsq_state_alloc(ctypes.byref(cfg.c()), ctypes.byref(bufs), ctypes.byref(h)) == 0
    return h.value


def batch(**kw):
    d = dict(io=lsq.IO_BF16, qk_heads=2, seqs=3, tokens=10, q_stride=256, k_stride=256, v_stride=256,
             o_stride=256, q=FAKE, k=FAKE, v=FAKE, alpha=FAKE, beta=FAKE, o=FAKE, cu_seqlens=FAKE,
             slots=FAKE, fresh=None)
    d.update(kw)
    return _lib.lsq_token_batch(**d)


BAD = [(dict(io=3), 1), (dict(io=-1), 1), (dict(seqs=-1), 1), (dict(tokens=-1), 1), (dict(qk_heads=3), 1),
       (dict(qk_heads=0), 1), (dict(qk_heads=8), 1), (dict(q_stride=-256), 1), (dict(k_stride=-8), 1),
       (dict(v_stride=-1), 1), (dict(o_stride=255), 1), (dict(o_stride=0), 1), (dict(q=None), 1),
       (dict(k=None), 1), (dict(v=None), 1), (dict(alpha=None), 1), (dict(beta=None), 1), (dict(o=None), 1),
       (dict(q=FAKE + 8), 1), (dict(k=FAKE + 2), 1), (dict(q_stride=260), 1), (dict(k_stride=257), 1),
       (dict(v=FAKE + 1), 1), (dict(o=FAKE + 1), 1), (dict(beta=FAKE + 2), 1), (dict(alpha=FAKE + 2), 1),
       (dict(slots=FAKE + 2), 1), (dict(slots=None, seqs=5), 1), (dict(io=lsq.IO_F32, v=FAKE + 2), 1)]


@pytest.mark.parametrize("change,status", BAD, ids=lambda x: str(x))
def test_batches_are_refused(change, status):
    L = _lib.load()
    h = handle()
    b = batch(**change)
    n = ctypes.c_size_t(0)
    need = L.lsq_attend_workspace(h, ctypes.byref(b), ctypes.byref(n)) == 0 and n.value
    assert L.lsq_attend(h, ctypes.byref(b), FAKE if need else None, n.value, None) == status
    assert L.lsq_last_error() != b""
    if b.seqs >= 0:
        b.tokens = b.seqs if b.tokens >= 0 else b.tokens
        assert L.lsq_step_slots(h, ctypes.byref(b), None) == status
    lsq.lsq_state_free(h)


def test_other_refusals():
    L = _lib.load()
    h = handle()
    b = batch()
    assert L.lsq_attend(None, ctypes.byref(b), None, 0, None) == 1
    assert L.lsq_attend(h, None, None, 0, None) == 1
    assert L.lsq_step_slots(None, ctypes.byref(b), None) == 1
    assert L.lsq_step_slots(h, None, None) == 1
    assert L.lsq_step_slots(h, ctypes.byref(b), None) == 1                  # tokens != seqs
    assert L.lsq_attend(h, ctypes.byref(batch(cu_seqlens=None)), None, 0, None) == 1
    assert L.lsq_attend(h, ctypes.byref(batch(cu_seqlens=FAKE + 1)), None, 0, None) == 1
    assert L.lsq_attend_workspace(h, ctypes.byref(b), None) == 1
    assert L.lsq_attend_workspace(None, ctypes.byref(b), ctypes.byref(ctypes.c_size_t())) == 1
    lsq.lsq_state_free(h)
    q = handle(bits=4, group=32, policy=lsq.POLICY_DYNAMIC)
    assert L.lsq_attend(q, ctypes.byref(b), None, 0, None) == 2             # a quantised handle
    assert L.lsq_step_slots(q, ctypes.byref(batch(tokens=3)), None) == 2
    lsq.lsq_state_free(q)
    d = handle(decay=lsq.DECAY_DIAG)
    assert L.lsq_step_slots(d, ctypes.byref(batch(tokens=3, alpha=FAKE + 4)), None) == 1
    lsq.lsq_state_free(d)


def test_attend_workspace():
    """Few tokens need none; many need a bounded one, which is checked."""
    L = _lib.load()
    h = handle()
    n = ctypes.c_size_t(1)
    need = lambda b: (L.lsq_attend_workspace(h, ctypes.byref(b), ctypes.byref(n)), n.value)[1]
    assert need(batch(tokens=1000, seqs=1)) == 0
    assert need(batch(tokens=0)) == 0
    one = need(batch(tokens=100_000, seqs=1))
    assert 0 < one <= need(batch(tokens=100_000, seqs=1000)) <= 64 << 20
    b = batch(tokens=100_000, seqs=1)
    assert L.lsq_attend(h, ctypes.byref(b), None, 0, None) == 1
    assert L.lsq_attend(h, ctypes.byref(b), None, one, None) == 1
    assert L.lsq_attend(h, ctypes.byref(b), FAKE + 4, one, None) == 1
    assert L.lsq_attend(h, ctypes.byref(b), FAKE, one - 1, None) == 3
    far = 16 << 20                                       # elements: 32 MiB between tokens
    for name in ("q_stride", "k_stride", "v_stride", "o_stride"):
        assert L.lsq_attend(h, ctypes.byref(batch(tokens=100, **{name: far})), None, 0, None) == 2
    lsq.lsq_state_free(h)
    for kw in (dict(delta=1), dict(decay=lsq.DECAY_DIAG)):   # token by token: none
        h = handle(**kw)
        assert need(batch(tokens=100_000, seqs=1)) == 0
        lsq.lsq_state_free(h)


def test_nothing_to_do_needs_no_pointers():
    L = _lib.load()
    h = handle()
    none = dict(q=None, k=None, v=None, alpha=None, beta=None, o=None, cu_seqlens=None, slots=None)
    for kw in (dict(seqs=0), dict(tokens=0), dict(seqs=0, tokens=0)):
        assert L.lsq_attend(h, ctypes.byref(batch(**none, **kw)), None, 0, None) == 0
    assert L.lsq_step_slots(h, ctypes.byref(batch(**none, seqs=0, tokens=0)), None) == 0
    lsq.lsq_state_free(h)
    e = handle(batch=0)
    assert L.lsq_attend(e, ctypes.byref(batch(**none)), None, 0, None) == 0
    lsq.lsq_state_free(e)
    e = handle(heads=0)
    assert L.lsq_attend(e, ctypes.byref(batch(**{**none, "qk_heads": 0})), None, 0, None) == 0
    lsq.lsq_state_free(e)


@pytest.mark.parametrize("fn,first,second", [("lsq_state_store_slots", "q", "f"), ("lsq_state_load_slots", "f", "q")])
def test_slot_copies_are_refused(fn, first, second):
    L = _lib.load()
    call = getattr(L, fn)
    h = {"f": handle(), "q": handle(bits=4, group=32, policy=lsq.POLICY_DYNAMIC)}
    a, b = h[first], h[second]
    assert call(None, b, 1, FAKE, FAKE, None) == 1
    assert call(a, None, 1, FAKE, FAKE, None) == 1
    assert call(a, b, -1, FAKE, FAKE, None) == 1
    assert call(b, a, 1, FAKE, FAKE, None) == 2                              # roles exchanged
    assert call(a, a, 1, FAKE, FAKE, None) == 2
    assert call(a, b, 1, FAKE + 2, FAKE, None) == 1
    assert call(a, b, 1, FAKE, FAKE + 2, None) == 1
    assert call(a, b, 5, None, FAKE, None) == 1                              # more entries than slots
    assert call(a, b, 5, FAKE, None, None) == 1
    assert call(a, b, 0, None, None, None) == 0
    for kw in (dict(heads=2), dict(dv=32), dict(dk=64)):
        other = handle(bits=4, group=32, policy=lsq.POLICY_DYNAMIC, **kw)
        x, y = (other, h["f"]) if first == "q" else (h["f"], other)
        assert call(x, y, 1, FAKE, FAKE, None) == 1
        lsq.lsq_state_free(other)
    lrb = handle(bits=4, group=32, policy=lsq.POLICY_DYNAMIC, lrb_rank=2)
    x, y = (lrb, h["f"]) if first == "q" else (h["f"], lrb)
    assert call(x, y, 1, FAKE, FAKE, None) == 2
    for x in (*h.values(), lrb):
        lsq.lsq_state_free(x)


def test_python_checks():
    """The binding's checks of tensors, on an object without device buffers."""
    st = object.__new__(lsq.LsqState)
    st.cfg = lsq.LsqConfig(batch=4, heads=4, dk=64, dv=32, bits=32, group=1, policy=lsq.POLICY_NONE)
    st.f32, st.codes = torch.empty(16, 32, 64), None
    n, bf = 5, torch.bfloat16
    good = dict(q=torch.zeros(n, 2, 64, dtype=bf), k=torch.zeros(n, 2, 64, dtype=bf),
                v=torch.zeros(n, 4, 32, dtype=bf), alpha=torch.zeros(n, 4), beta=torch.zeros(n, 4),
                cu_seqlens=torch.zeros(4, dtype=torch.int32), slots=torch.zeros(3, dtype=torch.int32),
                fresh=torch.zeros(3, dtype=torch.bool), o=None)
    b, o = slots.token_batch(st, **good)
    assert (b.io, b.qk_heads, b.seqs, b.tokens) == (lsq.IO_BF16, 2, 3, n)
    assert (b.q_stride, b.v_stride, b.o_stride) == (128, 128, 128) and o.shape == (n, 4, 32)
    wide = torch.zeros(n, 4 * 32 + 24, dtype=bf)
    b, _ = slots.token_batch(st, **{**good, "v": wide[:, :128].unflatten(1, (4, 32))})
    assert b.v_stride == 152
    b, _ = slots.token_batch(st, **{**good, "q": torch.zeros(1, 2, 64, dtype=bf).expand(n, 2, 64)})
    assert b.q_stride == 0
    for name, t in [("q", torch.zeros(n, 3, 64, dtype=bf)), ("q", torch.zeros(n, 2, 32, dtype=bf)),
                    ("q", torch.zeros(n, 128, dtype=bf)), ("q", torch.zeros(n, 2, 64, dtype=torch.float64)),
                    ("k", torch.zeros(n, 2, 64)), ("k", torch.zeros(n, 64, 2, dtype=bf).transpose(1, 2)),
                    ("v", torch.zeros(n, 2, 32, dtype=bf)), ("v", torch.zeros(n, 4, 64, dtype=bf)[:, :, ::2]),
                    ("alpha", torch.zeros(n, 4, dtype=bf)), ("alpha", torch.zeros(n, 4, 64)),
                    ("alpha", torch.zeros(4, n).t()), ("beta", torch.zeros(n, 2)),
                    ("cu_seqlens", torch.zeros(4, dtype=torch.int64)), ("cu_seqlens", torch.zeros(0, dtype=torch.int32)),
                    ("slots", torch.zeros(3, dtype=torch.int64)), ("slots", torch.zeros(2, dtype=torch.int32)),
                    ("fresh", torch.zeros(3)), ("fresh", torch.zeros(2, dtype=torch.bool)),
                    ("o", torch.zeros(n, 4, 32)), ("o", torch.zeros(n, 4, 31, dtype=bf))]:
        with pytest.raises(ValueError):
            slots.token_batch(st, **{**good, name: t})
    with pytest.raises(TypeError):
        st.store_slots(None)
    st.handle = None


def test_launches_of_too_many_threads_are_refused():
    """One launch holds fewer than 2^32 threads; nothing is launched."""
    L = _lib.load()
    h, q = handle(), handle(bits=4, group=32, policy=lsq.POLICY_DYNAMIC)
    n = 1 << 23                                             # entries: 2^25 blocks and more
    b = ctypes.byref(batch(seqs=n, tokens=n))
    assert L.lsq_step_slots(h, b, None) == 2
    assert L.lsq_attend(h, ctypes.byref(batch(seqs=n, tokens=100)), None, 0, None) == 2
    assert L.lsq_state_store_slots(q, h, n, FAKE, FAKE, None) == 2
    assert L.lsq_state_load_slots(h, q, n, FAKE, FAKE, None) == 2
    lsq.lsq_state_free(q)
    q = handle(bits=4, group=0, policy=lsq.POLICY_DYNAMIC)  # a block per head
    assert L.lsq_state_store_slots(q, h, n, FAKE, FAKE, None) == 2
    lsq.lsq_state_free(q)
    lsq.lsq_state_free(h)
