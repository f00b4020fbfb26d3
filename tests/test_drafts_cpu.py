"""Refusals of the drafted-token calls (no GPU needed, no kernel launched), and what the tests'
verification reference is for: the target's distribution.

The device pointers are never dereferenced: every call fails its checks, or has nothing to do, before
any launch.
"""
import ctypes
import itertools

import pytest
import torch

import quantized_recurrent_state_amd as lsq
from quantized_recurrent_state_amd import _lib, drafts
from tests.drafts_ref import residual
from tests.test_slots_cpu import BAD, FAKE, batch, handle


def tree(h, b, parents=FAKE, max_nodes=64):
    return _lib.load().lsq_step_tree(h, ctypes.byref(b), parents, max_nodes, None)


def accept(h, b, path=FAKE, lengths=FAKE, depth=4):
    return _lib.load().lsq_accept_path(h, ctypes.byref(b), path, lengths, depth, None)


@pytest.mark.parametrize("change,status", BAD, ids=lambda x: str(x))
def test_batches_are_refused(change, status):
    h, b = handle(), batch(**change)
    assert tree(h, b) == status
    if not set(change) <= {"q", "o", "q_stride", "o_stride"}:    # a path uses neither
        assert accept(h, b) == status
    assert _lib.load().lsq_last_error() != b""
    lsq.lsq_state_free(h)


def test_other_refusals():
    L, h, b = _lib.load(), handle(), batch()
    assert tree(None, b) == 1 and accept(None, b) == 1
    assert L.lsq_step_tree(h, None, FAKE, 64, None) == 1
    assert L.lsq_accept_path(h, None, FAKE, FAKE, 4, None) == 1
    for n, status in ((0, 1), (-1, 1), (65, 2), (1 << 30, 2)):
        assert tree(h, b, max_nodes=n) == status
    for n, status in ((-1, 1), (65, 2)):
        assert accept(h, b, depth=n) == status
    for p in (None, FAKE + 2):
        assert tree(h, b, parents=p) == 1
        assert accept(h, b, path=p) == 1 and accept(h, b, lengths=p) == 1
    assert tree(h, batch(cu_seqlens=None)) == 1 and accept(h, batch(cu_seqlens=None)) == 1
    assert tree(h, batch(cu_seqlens=FAKE + 1)) == 1 and accept(h, batch(cu_seqlens=FAKE + 1)) == 1
    lsq.lsq_state_free(h)
    q = handle(bits=4, group=32, policy=lsq.POLICY_DYNAMIC)
    assert tree(q, b) == 2 and accept(q, b) == 2
    lsq.lsq_state_free(q)
    d = handle(decay=lsq.DECAY_DIAG)
    assert tree(d, batch(alpha=FAKE + 4)) == 1 and accept(d, batch(alpha=FAKE + 4)) == 1
    lsq.lsq_state_free(d)


def test_nothing_to_do_needs_no_pointers():
    h = handle()
    none = dict(q=None, k=None, v=None, alpha=None, beta=None, o=None, cu_seqlens=None, slots=None)
    for kw in (dict(seqs=0), dict(tokens=0), dict(seqs=0, tokens=0)):
        assert tree(h, batch(**none, **kw), parents=None) == 0
        assert accept(h, batch(**none, **kw), path=None, lengths=None) == 0
    assert accept(h, batch(**none), path=None, lengths=None, depth=0) == 0
    lsq.lsq_state_free(h)
    for kw in (dict(batch=0), dict(heads=0)):
        e = handle(**kw)
        b = batch(**{**none, "qk_heads": 0 if "heads" in kw else 2})
        assert tree(e, b, parents=None) == 0 and accept(e, b, path=None, lengths=None) == 0
        lsq.lsq_state_free(e)


def draft(**kw):
    d = dict(seqs=3, vocab=1000, depth=8, replacement=1, nodes=10, target_stride=1000, draft_stride=1000)
    d.update({x: FAKE for x in ("target", "draft", "ids", "parents", "cu_nodes", "uniform", "uniform_next", "path",
                                "lengths", "next")})
    d.update(kw)
    return _lib.lsq_draft_batch(**d)


@pytest.mark.parametrize("change,status", [
    (dict(seqs=-1), 1), (dict(nodes=-1), 1), (dict(vocab=0), 1), (dict(vocab=-5), 1), (dict(depth=0), 1),
    (dict(replacement=2), 1), (dict(replacement=-1), 1), (dict(target_stride=-1), 1), (dict(draft_stride=-1), 1),
    (dict(vocab=(1 << 22) + 1), 2), (dict(seqs=1 << 22), 2),
    *[({x: None}, 1) for x in ("target", "ids", "parents", "cu_nodes", "uniform", "uniform_next", "path", "lengths", "next")],
    *[({x: FAKE + 2}, 1) for x in ("target", "draft", "ids", "parents", "cu_nodes", "uniform", "uniform_next", "path",
                                   "lengths", "next")]], ids=lambda x: str(x))
def test_draft_batches_are_refused(change, status):
    L = _lib.load()
    assert L.lsq_verify_tree(ctypes.byref(draft(**change)), FAKE, 1 << 40, None) == status
    assert L.lsq_last_error() != b""


def test_no_entries_to_verify():
    L = _lib.load()
    assert L.lsq_verify_tree(None, None, 0, None) == 1
    n = ctypes.c_size_t()
    assert L.lsq_verify_workspace(None, ctypes.byref(n)) == 1
    assert L.lsq_verify_workspace(ctypes.byref(draft()), None) == 1
    none = {x: None for x in ("target", "draft", "ids", "parents", "cu_nodes", "uniform", "uniform_next", "path",
                              "lengths", "next")}
    assert L.lsq_verify_tree(ctypes.byref(draft(seqs=0, **none)), None, 0, None) == 0


def test_verify_workspace():
    """Small vocabularies need none; larger ones a bounded one, which is checked."""
    L, n = _lib.load(), ctypes.c_size_t(1)
    need = lambda **kw: (L.lsq_verify_workspace(ctypes.byref(draft(**kw)), ctypes.byref(n)), n.value)[1]
    assert need(vocab=65536) == 0 and need(seqs=0, vocab=100_000) == 0
    for kw in (dict(vocab=65537), dict(vocab=131_072), dict(vocab=131_073, draft=None), dict(vocab=1 << 22, nodes=99)):
        size = need(**kw)
        assert 0 < size <= 3 * 4 * (kw["vocab"] // 128 + 2048)
        b = ctypes.byref(draft(**kw))
        assert L.lsq_verify_tree(b, None, size, None) == 1
        assert L.lsq_verify_tree(b, FAKE + 8, size, None) == 1
        assert L.lsq_verify_tree(b, FAKE, size - 1, None) == 3


def test_launches_of_too_many_threads_are_refused():
    h, n = handle(), 1 << 23
    assert tree(h, batch(seqs=n, tokens=100)) == 2
    assert accept(h, batch(seqs=n, tokens=100)) == 2
    lsq.lsq_state_free(h)


def _state():
    st = object.__new__(lsq.LsqState)
    st.cfg = lsq.LsqConfig(batch=4, heads=4, dk=64, dv=32, bits=32, group=1, policy=lsq.POLICY_NONE)
    st.f32, st.codes, st.handle = torch.empty(16, 32, 64), None, None
    return st


def test_python_checks(monkeypatch):
    """The binding's checks of tensors, on host tensors: nothing reaches the library."""
    st, n, m = _state(), 5, 3
    monkeypatch.setattr(drafts, "_on_device", lambda index, stream, call: call(0))
    monkeypatch.setattr(_lib, "load", lambda: pytest.fail("a call with bad tensors went through"))
    bf, i32 = torch.bfloat16, torch.int32
    good = dict(q=torch.zeros(n, 2, 64, dtype=bf), k=torch.zeros(n, 2, 64, dtype=bf), v=torch.zeros(n, 4, 32, dtype=bf),
                alpha=torch.zeros(n, 4), beta=torch.zeros(n, 4), cu_nodes=torch.zeros(m + 1, dtype=i32))
    for name, t in [("q", torch.zeros(n, 3, 64, dtype=bf)), ("k", torch.zeros(n, 2, 64)), ("cu_nodes", None),
                    ("cu_nodes", torch.zeros(m + 1)), ("parents", None), ("parents", torch.zeros(n)),
                    ("parents", torch.zeros(n + 1, dtype=i32)), ("slots", torch.zeros(m + 1, dtype=i32)),
                    ("fresh", torch.zeros(m)), ("o", torch.zeros(n, 4, 32))]:
        with pytest.raises(ValueError):
            st.step_tree(**{**good, "parents": torch.zeros(n, dtype=i32), name: t})
    path = dict(good, path=torch.zeros(m, 2, dtype=i32), lengths=torch.zeros(m, dtype=i32))
    del path["q"]
    for name, t in [("k", torch.zeros(n, 3, 64, dtype=bf)), ("k", torch.zeros(n, 128, dtype=bf)),
                    ("k", torch.zeros(n, 2, 64, dtype=torch.float64)), ("v", torch.zeros(n, 4, 32)), ("cu_nodes", None),
                    ("path", torch.zeros(m, dtype=i32)), ("path", torch.zeros(m + 1, 2, dtype=i32)),
                    ("path", torch.zeros(m, 2)), ("path", torch.zeros(m, 4, dtype=i32)[:, ::2]),
                    ("lengths", torch.zeros(m + 1, dtype=i32)), ("lengths", torch.zeros(m)),
                    ("slots", torch.zeros(m, dtype=torch.int64))]:
        with pytest.raises(ValueError):
            st.accept_path(**{**path, name: t})


def test_python_checks_of_verify():
    n, m, V = 5, 3, 40
    good = dict(target=torch.zeros(n, V), tokens=torch.zeros(n, dtype=torch.int32),
                parents=torch.zeros(n, dtype=torch.int32), cu_nodes=torch.zeros(m + 1, dtype=torch.int32),
                uniform=torch.zeros(n), uniform_next=torch.zeros(m), draft=torch.zeros(n, V), replacement=True, depth=7)
    b, ws, nb, path, lengths, token = drafts.draft_batch(**good)
    assert nb == 0                                       # a small vocabulary
    assert (b.seqs, b.vocab, b.depth, b.nodes, b.target_stride) == (m, V, 7, n, V)
    assert path.shape == (m, 7) and lengths.shape == (m,) and token.shape == (m,)
    wide = torch.zeros(n, V + 9)
    b, *_ = drafts.draft_batch(**{**good, "target": wide[:, :V], "draft": None})
    assert b.target_stride == V + 9 and b.draft is None
    b, *_ = drafts.draft_batch(**{**good, "draft": torch.zeros(1, V).expand(n, V)})
    assert b.draft_stride == 0
    for name, t in [("target", torch.zeros(n * V)), ("target", torch.zeros(n, V, dtype=torch.bfloat16)),
                    ("target", torch.zeros(V, n).t()), ("draft", torch.zeros(n, V + 1)), ("draft", torch.zeros(n, 2 * V)[:, ::2]),
                    ("tokens", torch.zeros(n, dtype=torch.int64)), ("parents", torch.zeros(n + 1, dtype=torch.int32)),
                    ("cu_nodes", torch.zeros(0, dtype=torch.int32)), ("cu_nodes", torch.zeros(m + 1)),
                    ("uniform", torch.zeros(n, dtype=torch.float64)), ("uniform_next", torch.zeros(m + 1)), ("depth", 0)]:
        with pytest.raises(ValueError):
            drafts.draft_batch(**{**good, name: t})
    with pytest.raises(ValueError):
        lsq.verify_tree(*(good[x] for x in ("target", "tokens", "parents", "cu_nodes", "uniform", "uniform_next")))


@pytest.mark.parametrize("drawn", ["with", "without", "given"])
def test_the_rule_keeps_the_targets_distribution(drawn):
    """Two children of one node, every pair of tokens they may have: the token behind the node (an
    accepted child, or the one drawn) has the target's distribution.  64 bits, by summation."""
    g = torch.Generator().manual_seed(5)
    for V in (2, 3, 5):
        p = torch.rand(V, generator=g, dtype=torch.float64)
        q = torch.rand(V, generator=g, dtype=torch.float64)
        p, q = p / p.sum(), q / q.sum()
        total = torch.zeros(V, dtype=torch.float64)
        for x, y in itertools.product(range(V), repeat=2):
            if drawn == "with":
                chance = float(q[x] * q[y])
            elif x == y:
                continue
            elif drawn == "without":
                chance = float(q[x] * q[y] / (1 - q[x]))
            else:                                        # certain drafts: each pair as likely as any
                chance = 1.0 / (V * (V - 1))
            rows = None if drawn == "given" else q
            left, reach = p, chance
            for n, t in enumerate((x, y)):
                left, gone = residual(p, rows, (x, y)[:n], drawn == "with")
                qt = 1.0 if rows is None else float(q[t]) / (1.0 if drawn == "with" else 1 - gone)
                take = min(1.0, float(left[t]) / qt)
                total[t] += reach * take
                reach *= 1 - take
            left, _ = residual(p, rows, (x, y), drawn == "with")
            total += reach * left / left.sum() if float(left.sum()) else 0.0
        assert float((total - p).abs().max()) < 1e-12


@pytest.mark.skipif(torch.cuda.device_count() > 0, reason="its made-up addresses must not reach a GPU")
@pytest.mark.parametrize("name", ["q_stride", "k_stride", "v_stride", "o_stride"])
def test_a_tree_of_far_rows_is_refused(name):
    """Strides below 2^31 elements pass every check and end with the launch's own error (HIP) on a host
    without a GPU; an accepted path takes any."""
    h = handle()
    for stride, status in (((1 << 31) - 8, 5), (1 << 31, 2), (1 << 40, 2), ((1 << 63) - 256, 2)):
        b = batch(**{name: stride})
        assert tree(h, b) == status, stride
        assert accept(h, b) == 5
    lsq.lsq_state_free(h)


def test_results_of_verify_do_not_hold_its_workspace():
    n, m, depth = 5, 3, 7
    for V in (40, 70_000):
        good = dict(target=torch.zeros(n, V), tokens=torch.zeros(n, dtype=torch.int32),
                    parents=torch.zeros(n, dtype=torch.int32), cu_nodes=torch.zeros(m + 1, dtype=torch.int32),
                    uniform=torch.zeros(n), uniform_next=torch.zeros(m), draft=torch.zeros(n, V), replacement=True, depth=depth)
        b, ws, nb, *results = drafts.draft_batch(**good)
        assert (nb > 0) == (V > 65536)
        for t, address, shape in zip(results, (b.path, b.lengths, b.next), ((m, depth), (m,), (m,))):
            assert t.dtype == torch.int32 and t.shape == shape and t.data_ptr() == address and t.is_contiguous()
            assert t.untyped_storage().nbytes() == 4 * m * (depth + 2)


def test_numbers_beyond_32_bits_do_not_wrap(monkeypatch):
    """The binding passes 32-bit numbers: 2^32 + 16 is no 16."""
    st, n, m, V = _state(), 5, 3, 40
    st.handle = h = handle(batch=4, heads=4, dk=64, dv=32)
    monkeypatch.setattr(drafts, "_on_device", lambda index, stream, call: call(0))
    x = dict(q=torch.zeros(n, 2, 64), k=torch.zeros(n, 2, 64), v=torch.zeros(n, 4, 32), alpha=torch.zeros(n, 4),
             beta=torch.zeros(n, 4), cu_nodes=torch.zeros(m + 1, dtype=torch.int32), parents=torch.zeros(n, dtype=torch.int32))
    for most, status in ((65, 2), ((1 << 32) + 16, 2), ((1 << 31) + 16, 2), (0, 1), (-(1 << 32) + 16, 1)):
        with pytest.raises(lsq.LsqError) as e:
            st.step_tree(**x, max_nodes=most)
        assert e.value.status == status
    lsq.lsq_state_free(h)
    good = dict(target=torch.zeros(n, V), tokens=torch.zeros(n, dtype=torch.int32),
                parents=torch.zeros(n, dtype=torch.int32), cu_nodes=torch.zeros(1, dtype=torch.int32),
                uniform=torch.zeros(n), uniform_next=torch.zeros(0), draft=None, replacement=True)
    for depth in (1 << 31, (1 << 32) + 7):               # no entries: nothing large is made here
        with pytest.raises(ValueError):
            drafts.draft_batch(**good, depth=depth)
    wide = torch.zeros(0, (1 << 32) + 5)                 # no rows
    none = {**good, "target": wide, "tokens": torch.zeros(0, dtype=torch.int32), "parents": torch.zeros(0, dtype=torch.int32),
            "uniform": torch.zeros(0)}
    with pytest.raises(lsq.LsqError) as e:
        drafts.draft_batch(**none, depth=7)
    assert e.value.status == 2
