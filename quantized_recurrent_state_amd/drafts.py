"""Tensor checks and calls of the drafted-token operators: ``LsqState.step_tree``, ``accept_path``
and ``verify_tree``."""
from __future__ import annotations

import ctypes

import torch

from . import _lib
from .slots import _buffer, _on_device, _plain, token_batch


def _i32(x):
    """x, or the nearest number that a 32-bit argument holds: the library refuses both alike."""
    return max(-2 ** 31, min(int(x), 2 ** 31 - 1))


def step_tree(state, q, k, v, alpha, beta, cu_nodes, parents, slots, fresh, max_nodes, o, stream):
    if cu_nodes is None or parents is None:
        raise ValueError("cu_nodes must hold seqs + 1 offsets, parents one entry per node")

    def call(s):
        b, out = token_batch(state, q, k, v, alpha, beta, cu_nodes, slots, fresh, o)
        pp = _plain("parents", parents, (b.tokens,), torch.int32, out.get_device())
        most = min(64, b.tokens or 1) if max_nodes is None else _i32(max_nodes)
        status = _lib.load().lsq_step_tree(state.handle, ctypes.byref(b), pp, most, s)
        if status:
            _lib.check(status, "lsq_step_tree")
        return out

    return _on_device(_buffer(state).get_device(), stream, call)


def accept_path(state, k, v, alpha, beta, cu_nodes, path, lengths, slots, fresh, stream):
    if cu_nodes is None:
        raise ValueError("cu_nodes must hold seqs + 1 offsets")
    if path.dim() != 2:
        raise ValueError(f"path has shape {tuple(path.shape)}, expected (seqs, depth)")

    def call(s):
        b, _ = token_batch(state, None, k, v, alpha, beta, cu_nodes, slots, fresh, None, outputs=False)
        dev, depth = k.get_device(), path.shape[1]
        pp = _plain("path", path, (b.seqs, depth), torch.int32, dev)
        lp = _plain("lengths", lengths, (b.seqs,), torch.int32, dev)
        status = _lib.load().lsq_accept_path(state.handle, ctypes.byref(b), pp, lp, depth, s)
        if status:
            _lib.check(status, "lsq_accept_path")

    _on_device(_buffer(state).get_device(), stream, call)


def _probabilities(name, t, shape, dev):
    """Address and row stride of an fp32 [nodes, vocab] tensor with contiguous rows."""
    if t.dtype is not torch.float32 or t.get_device() != dev:
        raise ValueError(f"{name} must be a float32 tensor on device {dev}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if not t.is_contiguous() and t.stride(1) != 1 and t.shape[1] != 1:
        raise ValueError(f"{name} must have contiguous rows")
    return t.data_ptr(), t.stride(0)


def draft_batch(target, tokens, parents, cu_nodes, uniform, uniform_next, draft, replacement, depth):
    """Checks the tensors of ``verify_tree``; returns (lsq_draft_batch, its workspace or None, the
    workspace's bytes, path, lengths, next)."""
    if target.dim() != 2:
        raise ValueError(f"target has shape {tuple(target.shape)}, expected (nodes, vocab)")
    if cu_nodes.dim() != 1 or cu_nodes.shape[0] < 1:
        raise ValueError("cu_nodes must hold seqs + 1 offsets")
    (n, vocab), dev, m, depth = target.shape, target.get_device(), cu_nodes.shape[0] - 1, int(depth)
    if not 1 <= depth < 2 ** 31:
        raise ValueError("depth must be at least 1, and below 2^31")
    tp, ts = _probabilities("target", target, (n, vocab), dev)
    dp, ds = (None, 0) if draft is None else _probabilities("draft", draft, (n, vocab), dev)
    ip = _plain("tokens", tokens, (n,), torch.int32, dev)
    pp = _plain("parents", parents, (n,), torch.int32, dev)
    cp = _plain("cu_nodes", cu_nodes, (m + 1,), torch.int32, dev)
    up = _plain("uniform", uniform, (n,), torch.float32, dev)
    np = _plain("uniform_next", uniform_next, (m,), torch.float32, dev)
    b = _lib.lsq_draft_batch(m, _i32(vocab), depth, 1 if replacement else 0, n, ts, ds, tp, dp, ip, pp, cp, up, np,
                             None, None, None)
    nb, ws = 0, None
    if vocab > 65536:                        # smaller rows need no workspace
        need = ctypes.c_size_t()
        status = _lib.load().lsq_verify_workspace(ctypes.byref(b), ctypes.byref(need))
        if status:
            _lib.check(status, "lsq_verify_workspace")
        nb = need.value
        ws = torch.empty(nb, dtype=torch.uint8, device=target.device) if nb else None
    # the outputs in one piece, apart from the workspace, which does not outlive the call
    buf = torch.empty(m * (depth + 2), dtype=torch.int32, device=target.device)
    at = buf.data_ptr()
    b.path, b.lengths, b.next = at, at + 4 * m * depth, at + 4 * m * (depth + 1)
    path, lengths, token = buf.split_with_sizes((m * depth, m, m))
    return b, ws, nb, path.view(m, depth), lengths, token


def verify_tree(target, tokens, parents, cu_nodes, uniform, uniform_next, draft, replacement, depth, stream):
    if not target.is_cuda:
        raise ValueError("target must be a device tensor")

    def call(s):
        b, ws, nb, path, lengths, token = draft_batch(target, tokens, parents, cu_nodes, uniform, uniform_next,
                                                      draft, replacement, depth)
        status = _lib.load().lsq_verify_tree(ctypes.byref(b), ws.data_ptr() if nb else None, nb, s)
        if status:
            _lib.check(status, "lsq_verify_tree")
        return path, lengths, token

    return _on_device(target.get_device(), stream, call)
