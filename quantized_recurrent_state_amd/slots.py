"""Tensor checks and calls of the slot operators behind ``LsqState``'s methods.

A decode step of one token is a few microseconds on the GPU, so the checks read each tensor
attribute once and the common case (the state's device current, its current stream) takes no
context manager.
"""
from __future__ import annotations

import ctypes

import torch

from . import DECAY_DIAG, IO_BF16, IO_F16, IO_F32, LsqState, _lib

_IO = {torch.float32: IO_F32, torch.float16: IO_F16, torch.bfloat16: IO_BF16}


# The current stream's address without the Stream object around it, where torch has the call.
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                          lambda index: torch.cuda.current_stream(index).cuda_stream)


def _buffer(state):
    return state.f32 if state.codes is None else state.codes


def _on_device(index, stream, call):
    """call(stream pointer) with the state's device current and, where a stream is given, with it
    current too: what is allocated in the call then belongs to it."""
    if stream is not None:
        if not isinstance(stream, torch.cuda.Stream):
            stream = torch.cuda.ExternalStream(int(stream), device=index)
        if stream.device.index != index:
            raise ValueError(f"stream is on device {stream.device.index}, the state on {index}")
        with torch.cuda.stream(stream):
            return call(stream.cuda_stream)
    if index == torch.cuda.current_device():
        return call(_current_stream(index))
    with torch.cuda.device(index):
        return call(_current_stream(index))


def _plain(name, t, shape, dtype, index):
    """Address of a contiguous tensor of this shape and type on device index."""
    if t.dtype is not dtype or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor on device {index}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    return t.data_ptr()


def _rows(name, t, shape, dtype, index):
    """Address and token stride of a [tokens, heads, d] tensor whose tokens may be strided."""
    if t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be a {dtype} tensor on device {index}")
    if t.shape != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    n, heads, d = shape
    if t.is_contiguous():                    # also one token of any stride
        return t.data_ptr(), heads * d
    row, head, one = t.stride()
    if (one != 1 and d != 1) or (head != d and heads != 1):
        raise ValueError(f"{name} must be contiguous within each token")
    return t.data_ptr(), row


def token_batch(state, q, k, v, alpha, beta, cu_seqlens, slots, fresh, o, outputs=True):
    """Checks a token batch's tensors; returns (lsq_token_batch, o).  outputs False: without q and o."""
    c = state.cfg
    if c.bits != 32:
        raise ValueError("token batches run on an fp32 state (bits 32)")
    first, name = (q, "q") if outputs else (k, "k")
    dev, dtype = state.f32.get_device(), first.dtype
    io = _IO.get(dtype)
    if io is None:
        raise ValueError(f"{name} has type {dtype}, expected float32, float16 or bfloat16")
    if first.dim() != 3:
        raise ValueError(f"{name} has shape {tuple(first.shape)}, expected (tokens, qk_heads, {c.dk})")
    n, hk, _ = first.shape
    heads, dk, dv = c.heads, c.dk, c.dv
    if hk == 0 or heads % hk:
        raise ValueError(f"{name} has {hk} heads, which must divide the state's {heads}")
    qp, sq = _rows("q", q, (n, hk, dk), dtype, dev) if outputs else (None, 0)
    kp, sk = _rows("k", k, (n, hk, dk), dtype, dev)
    vp, sv = _rows("v", v, (n, heads, dv), dtype, dev)
    ap = _plain("alpha", alpha, (n, heads, dk) if c.decay == DECAY_DIAG else (n, heads), torch.float32, dev)
    bp = _plain("beta", beta, (n, heads), torch.float32, dev)
    m, cp, sp, fp = n, None, None, None
    if cu_seqlens is not None:
        if cu_seqlens.dim() != 1 or cu_seqlens.shape[0] < 1:
            raise ValueError("cu_seqlens must hold seqs + 1 offsets")
        m = cu_seqlens.shape[0] - 1
        cp = _plain("cu_seqlens", cu_seqlens, (m + 1,), torch.int32, dev)
    if slots is not None:
        sp = _plain("slots", slots, (m,), torch.int32, dev)
    if fresh is not None:
        fp = _plain("fresh", fresh, (m,), torch.bool if fresh.dtype is torch.bool else torch.uint8, dev)
    if not outputs:
        op, so = None, 0
    elif o is None:
        o = torch.empty((n, heads, dv), dtype=dtype, device=state.f32.device)
        op, so = o.data_ptr(), heads * dv
    else:
        op, so = _rows("o", o, (n, heads, dv), dtype, dev)
    return _lib.lsq_token_batch(io, hk, m, n, sq, sk, sv, so, qp, kp, vp, ap, bp, op, cp, sp, fp), o


def attend(state, q, k, v, alpha, beta, cu_seqlens, slots, fresh, o, stream):
    if cu_seqlens is None:
        raise ValueError("cu_seqlens must hold seqs + 1 offsets")

    def call(s):
        lib = _lib.load()
        b, out = token_batch(state, q, k, v, alpha, beta, cu_seqlens, slots, fresh, o)
        nb, ws, status = 0, None, 0
        if b.tokens > 1024:                  # smaller batches need none
            need = ctypes.c_size_t()
            status = lib.lsq_attend_workspace(state.handle, ctypes.byref(b), ctypes.byref(need))
            nb = need.value
            ws = torch.empty(nb, dtype=torch.uint8, device=out.device) if nb else None
        if status == 0:
            status = lib.lsq_attend(state.handle, ctypes.byref(b), ws.data_ptr() if nb else None, nb, s)
        if status:
            _lib.check(status, "lsq_attend")
        return out

    return _on_device(_buffer(state).get_device(), stream, call)


def step_slots(state, q, k, v, alpha, beta, slots, fresh, o, stream):
    def call(s):
        b, out = token_batch(state, q, k, v, alpha, beta, None, slots, fresh, o)
        status = _lib.load().lsq_step_slots(state.handle, ctypes.byref(b), s)
        if status:
            _lib.check(status, "lsq_step_slots")
        return out

    return _on_device(_buffer(state).get_device(), stream, call)


def copy(fn, dst, src, dst_slots, src_slots, stream):
    """fn (lsq_state_store_slots or lsq_state_load_slots) of the entries that the slots list."""
    if not isinstance(dst, LsqState) or not isinstance(src, LsqState):
        raise TypeError("both states must be LsqState")
    dev = _buffer(dst).get_device()
    if _buffer(src).get_device() != dev:
        raise ValueError("both states must be on one device")
    m = min(dst.cfg.batch, src.cfg.batch)
    for t in (dst_slots, src_slots):
        if t is not None:
            m = t.shape[0]
    for name, t in (("dst_slots", dst_slots), ("src_slots", src_slots)):
        if t is not None:
            _plain(name, t, (m,), torch.int32, dev)
    _on_device(dev, stream, lambda s: fn(dst.handle, src.handle, m, dst_slots, src_slots, s))
