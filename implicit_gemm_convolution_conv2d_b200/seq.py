"""Sequence operators: the causal depthwise convolution, the gated linear
recurrence and 8-bit activation checkpoints (the C ABI in ``include/conv_seq.h``).

Tokens are rows of C channels, channels last.  A batch is [N, L, C]; sequences
of different lengths are packed end to end in [rows, C] with ``cu_seqlens``, a
CUDA int32 tensor of N + 1 non-decreasing offsets (empty sequences are allowed).
Rows in no sequence (behind the last one) are never read into a result; their
output rows are zero in a tensor that the call makes, and left as they are in
one that the caller passes as ``out``.  ``cu_seqlens`` and ``index`` are read on
the device and not checked: entries out of order or out of range give
unspecified results, but no access out of bounds.

Inputs may have any token and batch stride as long as a token's channels are
contiguous (the halves of a fused projection's output are taken as they are);
others are copied.  Like the convolutions, every call only queues its kernels,
on the current stream or on ``stream``; what it allocates belongs to that stream.
"""
from __future__ import annotations

import ctypes
import functools
from typing import NamedTuple

import torch

from . import CONV_BF16, CONV_F16, CONV_F32, ConvError, lib as _load

__all__ = ["conv_causal", "conv_causal_grad", "conv_causal_step", "gated_scan", "gated_scan_grad", "gated_scan_step",
           "Act8", "act8_pack", "act8_unpack", "GATED_SCAN_STATE_EVERY", "ACT8_BLOCK", "CONV_CAUSAL_MAX_K"]

GATED_SCAN_STATE_EVERY = 64
ACT8_BLOCK = 32
CONV_CAUSAL_MAX_K = 8
_DTYPE = {torch.float32: CONV_F32, torch.float16: CONV_F16, torch.bfloat16: CONV_BF16}
_ACT = {None: 0, "silu": 1}


class Act8(NamedTuple):
    """An activation in 8 bits: int8 values, the byte e + 127 of each 32 channels' step 2^e, and the type it had."""

    q: torch.Tensor
    scale: torch.Tensor
    dtype: torch.dtype

    @property
    def shape(self):
        return self.q.shape


_fn = {}


def _lib():
    """The library's sequence functions by name, their argument types set."""
    if not _fn:
        L = _load()
        p, i, n = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong
        size = [ctypes.c_ulonglong]
        out = [ctypes.POINTER(ctypes.c_ulonglong)]
        table = {}
        for name, args in {
            "conv_causal": [p] * 7 + [i, n, i, i, n, n, i, i, i, p],
            "conv_causal_grad": [p] * 12 + [i, n, i, i] + [n] * 4 + [i, i, i, p] + size + [p],
            "conv_causal_grad_workspace_size": [i, n, i, i, i] + out,
            "conv_causal_step": [p] * 6 + [i, i, i, i, n, i, i, i, p],
            "gated_scan": [p] * 9 + [i, n, i] + [n] * 6 + [i, i, p],
            "gated_scan_grad": [p] * 17 + [i, n, i] + [n] * 8 + [i, i, p] + size + [p],
            "gated_scan_grad_workspace_size": [i, n, i, i] + out,
            "gated_scan_step": [p] * 7 + [i, i, i, n, n, n, i, i, p],
            "act8_pack": [p, p, p, n, i, n, i, p],
            "act8_unpack": [p, p, p, n, i, i, p],
        }.items():
            f = getattr(L, name)
            f.argtypes, f.restype = args, i
            table[name] = f
        _fn.update(table)  # all at once: another thread may be looking
    return _fn


_current_device, _raw_stream = torch._C._cuda_getDevice, torch._C._cuda_getCurrentRawStream


def _elsewhere(t, stream):
    """A context that makes a call's stream, or its tensors' device, current; None where they are."""
    if stream is not None:
        if stream.device != t.device:
            raise ValueError(f"the stream is on {stream.device}, the tensors on {t.device}")
        return torch.cuda.stream(stream)
    if t.get_device() != _current_device():
        return torch.cuda.device(t.device)
    return None


def _new_like(t):
    """A contiguous tensor of t's shape and type (empty_like, where it gives that, costs the host least)."""
    return torch.empty_like(t) if t.is_contiguous() else t.new_empty(t.shape)


def _code(dtype, what):
    code = _DTYPE.get(dtype)
    if code is None:
        raise TypeError(f"{what}: unsupported dtype {dtype}")
    return code


def _cuda(t, name, what):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{what}: {name} must be a tensor")
    if not t.is_cuda:
        raise ValueError(f"{what} runs on CUDA tensors only ({name} is not one)")


def _same_device(like, what, names, *tensors):
    """Every tensor is on the device of `like`; `names` has their names, for the error."""
    at = like.get_device()
    for k, t in enumerate(tensors):
        if t is not None and not (isinstance(t, torch.Tensor) and t.get_device() == at):
            name = names.split()[k]
            _cuda(t, name, what)
            raise ValueError(f"{what}: {name} is on {t.device}, x on {like.device}")


def _fits(what, *sizes):
    """The library takes these as 32-bit integers, and ctypes would cut them off."""
    if max(sizes) > 0x7FFFFFFF:
        raise ValueError(f"{what}: sequences, rows of a step, slots and channels are at most 2^31 - 1, not {max(sizes)}")


def _extents(x, cu, what):
    """(N, L, C) of tokens: [N, L, C], or packed [L, C] with N sequences."""
    if cu is None:
        if x.dim() != 3:
            raise ValueError(f"{what}: without cu_seqlens x must be [N, L, C]")
        N, L, C = x.shape
    else:
        if x.dim() != 2:
            raise ValueError(f"{what}: with cu_seqlens x must be [rows, C]")
        if cu.dim() != 1 or cu.dtype != torch.int32 or cu.shape[0] < 1:
            raise ValueError(f"{what}: cu_seqlens must be int32 of N + 1 offsets")
        if not cu.is_contiguous():
            raise ValueError(f"{what}: cu_seqlens must be contiguous")
        L, C = x.shape
        N = cu.shape[0] - 1
    if C < 1:
        raise ValueError(f"{what}: x has no channels")
    _fits(what, N, C)
    return N, L, C


def _rows(t, packed):
    """t with contiguous channels, and its batch and token strides."""
    st = t.stride()
    if st[-1] != 1 and t.shape[-1] > 1:
        t = t.contiguous()
        st = t.stride()
    return (t, 0, st[0]) if packed else (t, st[0], st[1])


def _check(t, shape, dtype, name, what):
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{what}: {name} must be {dtype} of shape {tuple(shape)}, not {t.dtype} of {tuple(t.shape)}")


def _check_out(t, shape, dtype, name, what):
    _check(t, shape, dtype, name, what)
    if not t.is_contiguous():
        raise ValueError(f"{what}: {name} must be contiguous")


def _optional(t, shape, dtype, name, what):
    """An input of a fixed shape, contiguous; None stays None."""
    if t is None:
        return None
    _check(t, shape, dtype, name, what)
    return t.contiguous()


def _ptr(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=4096)
def _workspace(name, *sizes):
    """Bytes of workspace for these sizes, of which it is a function alone."""
    out = ctypes.c_ulonglong()
    _raise(_lib()[name](*sizes, ctypes.byref(out)), name)
    return out.value


def _raise(rc, what):
    if rc:
        raise ConvError(rc, what)


def _saved(v, what, name):
    """(values, scales or None, dtype) of an activation or its checkpoint."""
    if isinstance(v, Act8):
        _cuda(v.q, name, what)
        _same_device(v.q, what, "scale", v.scale)
        blocks = (v.q.shape[-1] + ACT8_BLOCK - 1) // ACT8_BLOCK if v.q.dim() else 0
        _check(v.q, v.q.shape, torch.int8, f"{name}.q", what)
        _check(v.scale, (*v.q.shape[:-1], blocks), torch.uint8, f"{name}.scale", what)
        return v.q, v.scale, v.dtype
    _cuda(v, name, what)
    return v, None, v.dtype


# ---- 8-bit activation checkpoints ---------------------------------------


def act8_pack(x, *, stream=None) -> Act8:
    """x [..., C] in 8 bits: blocks of 32 channels share a power of two, the
    least by which the block's largest magnitude is at most 127, and each element
    is rounded to the nearest multiple of it: off by at most half of it, or by less
    than one where that multiple would be past the type's largest value (65504 in
    float16 comes back as 64512).  A block with an infinity or NaN comes back as NaN."""
    what = "act8_pack"
    _cuda(x, "x", what)
    code = _code(x.dtype, what)
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError(f"{what}: x must be [..., C]")
    C = x.shape[-1]
    _fits(what, C)
    there = _elsewhere(x, stream)
    if there is not None:
        with there:
            return act8_pack(x)
    stream = _raw_stream(x.get_device())
    if x.dim() != 2 or x.stride(1) != 1 and C > 1:
        x = x.contiguous()
    rows = x.numel() // C
    q = torch.empty_like(x, dtype=torch.int8, memory_format=torch.contiguous_format)
    scale = x.new_empty((*x.shape[:-1], (C + ACT8_BLOCK - 1) // ACT8_BLOCK), dtype=torch.uint8)
    _raise(_lib()["act8_pack"](x.data_ptr(), q.data_ptr(), scale.data_ptr(), rows, C,
                               x.stride(0) if x.dim() == 2 else C, code, stream), what)
    return Act8(q, scale, x.dtype)


def act8_unpack(p: Act8, *, out=None, stream=None):
    """The activation that a checkpoint stands for, in the type it had."""
    what = "act8_unpack"
    if not isinstance(p, Act8):
        raise TypeError(f"{what}: takes an Act8")
    q, scale, dtype = _saved(p, what, "p")
    code = _code(dtype, what)
    if q.dim() < 1 or q.shape[-1] < 1:
        raise ValueError(f"{what}: p must be [..., C]")
    C = q.shape[-1]
    _fits(what, C)
    _same_device(q, what, "out", out)
    there = _elsewhere(q, stream)
    if there is not None:
        with there:
            return act8_unpack(p, out=out)
    stream = _raw_stream(q.get_device())
    if out is None:
        out = torch.empty_like(q, dtype=dtype, memory_format=torch.contiguous_format)
    else:
        _check_out(out, q.shape, dtype, "out", what)
    q, scale = q.contiguous(), scale.contiguous()
    _raise(_lib()["act8_unpack"](q.data_ptr(), scale.data_ptr(), out.data_ptr(), q.numel() // C, C, code,
                                 stream), what)
    return out


# ---- causal depthwise convolution ---------------------------------------


def _filter(x_dtype, C, w, bias, activation, what):
    if w.dim() != 2 or w.shape[0] != C or not 1 <= w.shape[1] <= CONV_CAUSAL_MAX_K:
        raise ValueError(f"{what}: w must be [C, K] with C = {C} and 1 <= K <= {CONV_CAUSAL_MAX_K}, not {tuple(w.shape)}")
    if w.dtype != x_dtype:
        raise TypeError(f"{what}: x and w must share a dtype")
    if activation not in _ACT:
        raise ValueError(f"{what}: activation must be None or 'silu'")
    return w.contiguous(), _optional(bias, (C,), x_dtype, "bias", what), w.shape[1]


def conv_causal(x, w, bias=None, *, activation=None, state=None, cu_seqlens=None, return_state=False, out=None,
                stream=None):
    """Depthwise convolution along time that sees no later token:
    y[t, c] = act(bias[c] + sum_j w[c, j] * x[t - (K-1) + j, c]) in each sequence.

    x: [N, L, C] or packed [rows, C]; w: [C, K], K <= 8; activation: None or
    "silu".  `state` [N, K-1, C] holds the rows in front of each sequence (zeros
    without it).  Returns y, or with `return_state` (y, the window that continues
    each sequence)."""
    what = "conv_causal"
    _cuda(x, "x", what)
    _same_device(x, what, "w bias state cu_seqlens out", w, bias, state, cu_seqlens, out)
    code = _code(x.dtype, what)
    N, L, C = _extents(x, cu_seqlens, what)
    there = _elsewhere(x, stream)
    if there is not None:
        with there:
            return conv_causal(x, w, bias, activation=activation, state=state, cu_seqlens=cu_seqlens,
                               return_state=return_state, out=out)
    stream = _raw_stream(x.get_device())
    w, bias, K = _filter(x.dtype, C, w, bias, activation, what)
    state = _optional(state, (N, K - 1, C), x.dtype, "state", what)
    fill = out is None
    if fill:
        out = _new_like(x)
    else:
        _check_out(out, x.shape, x.dtype, "out", what)
    left = x.new_empty((N, K - 1, C)) if return_state else None
    x, xb, xt = _rows(x, cu_seqlens is not None)
    _raise(_lib()["conv_causal"](x.data_ptr(), w.data_ptr(), _ptr(bias), _ptr(state), _ptr(cu_seqlens),
                                 out.data_ptr(), _ptr(left), N, L, C, K, xb, xt, _ACT[activation], fill, code,
                                 stream), what)
    return (out, left) if return_state else out


def conv_causal_grad(x, w, dy, bias=None, *, activation=None, state=None, dstate_out=None, cu_seqlens=None,
                     stream=None):
    """Gradients of conv_causal: (dx, dw, dbias, dstate) from dy, the gradient of
    y, and `dstate_out`, that of the window it returned (if it matters).

    x may be the activation or its checkpoint (Act8).  dbias and dstate are None
    where the forward pass had no bias or state."""
    what = "conv_causal_grad"
    xv, xs, dtype = _saved(x, what, "x")
    _same_device(xv, what, "w dy bias state dstate_out cu_seqlens", w, dy, bias, state, dstate_out, cu_seqlens)
    code = _code(dtype, what)
    N, L, C = _extents(xv, cu_seqlens, what)
    _check(dy, xv.shape, dtype, "dy", what)
    packed = cu_seqlens is not None
    there = _elsewhere(xv, stream)
    if there is not None:
        with there:
            return conv_causal_grad(x, w, dy, bias, activation=activation, state=state, dstate_out=dstate_out,
                                    cu_seqlens=cu_seqlens)
    stream = _raw_stream(xv.get_device())
    w, bias, K = _filter(dtype, C, w, bias, activation, what)
    state = _optional(state, (N, K - 1, C), dtype, "state", what)
    dstate_out = _optional(dstate_out, (N, K - 1, C), dtype, "dstate_out", what)
    xv, xb, xt = _rows(xv, packed)
    dy, yb, yt = _rows(dy, packed)
    if xs is not None:
        xs = xs.contiguous()
    dx = _new_like(dy)
    dw = dy.new_empty((C, K))
    db = None if bias is None else dy.new_empty(C)
    ds = None if state is None else dy.new_empty((N, K - 1, C))
    need = _workspace("conv_causal_grad_workspace_size", N, L, C, K, packed)
    work = dy.new_empty(need // 4, dtype=torch.float32)
    _raise(_lib()["conv_causal_grad"](xv.data_ptr(), _ptr(xs), w.data_ptr(), _ptr(bias), _ptr(state),
                                      _ptr(cu_seqlens), dy.data_ptr(), _ptr(dstate_out), dx.data_ptr(),
                                      dw.data_ptr(), _ptr(db), _ptr(ds), N, L, C, K, xb, xt, yb, yt,
                                      _ACT[activation], True, code, work.data_ptr(), need, stream), what)
    return dx, dw, db, ds


def _step_rows(x, pool_rows, index, what):
    if x.dim() != 2 or x.shape[1] < 1:
        raise ValueError(f"{what}: x must be [B, C]")
    B = x.shape[0]
    _fits(what, B, pool_rows, x.shape[1])
    if index is None:
        if B > pool_rows:
            raise ValueError(f"{what}: {B} rows but {pool_rows} slots: give an index")
    elif tuple(index.shape) != (B,) or index.dtype != torch.int32 or not index.is_contiguous():
        raise ValueError(f"{what}: index must be a contiguous int32 of shape ({B},)")
    return B


def conv_causal_step(x, w, state, bias=None, *, activation=None, index=None, out=None, stream=None):
    """conv_causal for one token of each of B sequences: x [B, C] -> y [B, C].

    `state` [slots, K-1, C] holds the sequences' windows and is updated in place.
    Row b uses slot index[b] (int32; slot b without an index).  A row whose index
    is negative or past the slots is skipped: its y row is zero, or left as it is
    in a given `out`.  Rows naming one slot are taken in row order, as that
    sequence's consecutive tokens."""
    what = "conv_causal_step"
    _cuda(x, "x", what)
    _same_device(x, what, "w state bias index out", w, state, bias, index, out)
    code = _code(x.dtype, what)
    B, C = _step_rows(x, state.shape[0] if state.dim() == 3 else 0, index, what), x.shape[1]
    there = _elsewhere(x, stream)
    if there is not None:
        with there:
            return conv_causal_step(x, w, state, bias, activation=activation, index=index, out=out)
    stream = _raw_stream(x.get_device())
    w, bias, K = _filter(x.dtype, C, w, bias, activation, what)
    slots = state.shape[0]
    _check_out(state, (slots, K - 1, C), x.dtype, "state", what)
    fill = out is None
    if fill:
        out = _new_like(x)
    else:
        _check_out(out, x.shape, x.dtype, "out", what)
    x, _, xt = _rows(x, True)
    _raise(_lib()["conv_causal_step"](x.data_ptr(), w.data_ptr(), _ptr(bias), state.data_ptr(), _ptr(index),
                                      out.data_ptr(), B, slots, C, K, xt, _ACT[activation], fill, code,
                                      stream), what)
    return out


# ---- gated linear recurrence --------------------------------------------


def _decay(decay, C, what):
    _check(decay, (C,), torch.float32, "decay", what)
    return decay.contiguous()


def gated_scan(x, r, i, decay, *, h0=None, cu_seqlens=None, save_states=False, out=None, stream=None):
    """The gated linear recurrence of each channel along each sequence:
    a = exp(-decay * sigmoid(r)), h[t] = a h[t-1] + sqrt(1 - a^2) sigmoid(i) x[t], y = h.

    x, r, i: [N, L, C] or packed [rows, C]; decay: [C] fp32, not negative; h0:
    [N, C] fp32 (zeros without it).  Returns (y, h_last [N, C] fp32), and with
    `save_states` also the states that gated_scan_grad starts from: those in
    front of every 64th token, fp32 [N, ceil(L / 64), C] (packed: N = 1)."""
    what = "gated_scan"
    _cuda(x, "x", what)
    _same_device(x, what, "r i decay h0 cu_seqlens out", r, i, decay, h0, cu_seqlens, out)
    code = _code(x.dtype, what)
    N, L, C = _extents(x, cu_seqlens, what)
    _check(r, x.shape, x.dtype, "r", what)
    _check(i, x.shape, x.dtype, "i", what)
    packed = cu_seqlens is not None
    there = _elsewhere(x, stream)
    if there is not None:
        with there:
            return gated_scan(x, r, i, decay, h0=h0, cu_seqlens=cu_seqlens, save_states=save_states, out=out)
    stream = _raw_stream(x.get_device())
    decay = _decay(decay, C, what)
    h0 = _optional(h0, (N, C), torch.float32, "h0", what)
    fill = out is None
    if fill:
        out = _new_like(x)
    else:
        _check_out(out, x.shape, x.dtype, "out", what)
    last = decay.new_empty((N, C))
    states = None
    if save_states:
        states = decay.new_empty((1 if packed else N, (L + 63) // 64, C))
    x, xb, xt = _rows(x, packed)
    r, rb, rt = _rows(r, packed)
    i, ib, it = _rows(i, packed)
    _raise(_lib()["gated_scan"](x.data_ptr(), r.data_ptr(), i.data_ptr(), decay.data_ptr(), _ptr(h0),
                                _ptr(cu_seqlens), out.data_ptr(), last.data_ptr(), _ptr(states), N, L, C, xb, xt,
                                rb, rt, ib, it, fill, code, stream), what)
    return (out, last, states) if save_states else (out, last)


def gated_scan_grad(x, r, i, decay, dy, states, *, h0=None, dh_last=None, cu_seqlens=None, stream=None):
    """Gradients of gated_scan: (dx, dr, di, ddecay, dh0) from dy, the gradient of
    y, and `dh_last`, that of the last states (if it matters).

    x, r and i may each be the activation or its checkpoint (Act8; a mixture is
    unpacked into temporaries); `states` are the forward pass's.  ddecay and dh0 are
    fp32; dh0 is None without h0."""
    what = "gated_scan_grad"
    xv, xs, dtype = _saved(x, what, "x")
    rv, rs, rd = _saved(r, what, "r")
    iv, is_, idt = _saved(i, what, "i")
    _same_device(xv, what, "r i decay dy states h0 dh_last cu_seqlens", rv, iv, decay, dy, states, h0, dh_last, cu_seqlens)
    code = _code(dtype, what)
    N, L, C = _extents(xv, cu_seqlens, what)
    for name, t, d in (("r", rv, rd), ("i", iv, idt), ("dy", dy, dy.dtype)):
        if t.shape != xv.shape or d != dtype:
            raise ValueError(f"{what}: {name} must be {dtype} of shape {tuple(xv.shape)}")
    packed = cu_seqlens is not None
    there = _elsewhere(xv, stream)
    if there is not None:
        with there:
            return gated_scan_grad(x, r, i, decay, dy, states, h0=h0, dh_last=dh_last, cu_seqlens=cu_seqlens)
    stream = _raw_stream(xv.get_device())
    if not (xs is None) == (rs is None) == (is_ is None):  # a mixture: the kernel takes all or none in 8 bits
        xv, rv, iv = (act8_unpack(v) if isinstance(v, Act8) else v for v in (x, r, i))
        xs = rs = is_ = None
    decay = _decay(decay, C, what)
    states = _optional(states, (1 if packed else N, (L + 63) // 64, C), torch.float32, "states", what)
    h0 = _optional(h0, (N, C), torch.float32, "h0", what)
    dh_last = _optional(dh_last, (N, C), torch.float32, "dh_last", what)
    if xs is not None:
        xv, rv, iv, xs, rs, is_ = (t.contiguous() for t in (xv, rv, iv, xs, rs, is_))
    xv, xb, xt = _rows(xv, packed)
    rv, rb, rt = _rows(rv, packed)
    iv, ib, it = _rows(iv, packed)
    dy, yb, yt = _rows(dy, packed)
    dx, dr, di = _new_like(dy), _new_like(dy), _new_like(dy)
    ddecay = decay.new_empty(C)
    dh0 = None if h0 is None else decay.new_empty((N, C))
    need = _workspace("gated_scan_grad_workspace_size", N, L, C, packed)
    work = decay.new_empty(need // 4)
    _raise(_lib()["gated_scan_grad"](xv.data_ptr(), _ptr(xs), rv.data_ptr(), _ptr(rs), iv.data_ptr(), _ptr(is_),
                                     decay.data_ptr(), _ptr(states), _ptr(h0), _ptr(cu_seqlens), dy.data_ptr(),
                                     _ptr(dh_last), dx.data_ptr(), dr.data_ptr(), di.data_ptr(),
                                     ddecay.data_ptr(), _ptr(dh0), N, L, C, xb, xt, rb, rt, ib, it, yb, yt, True,
                                     code, work.data_ptr(), need, stream), what)
    return dx, dr, di, ddecay, dh0


def gated_scan_step(x, r, i, decay, h, *, index=None, out=None, stream=None):
    """gated_scan for one token of each of B sequences: x, r, i [B, C] -> y [B, C].

    `h` [slots, C] fp32 holds the states and is updated in place; `index`, skipped
    rows and rows naming one slot as for conv_causal_step."""
    what = "gated_scan_step"
    _cuda(x, "x", what)
    _same_device(x, what, "r i decay h index out", r, i, decay, h, index, out)
    code = _code(x.dtype, what)
    B, C = _step_rows(x, h.shape[0] if h.dim() == 2 else 0, index, what), x.shape[1]
    _check(r, x.shape, x.dtype, "r", what)
    _check(i, x.shape, x.dtype, "i", what)
    slots = h.shape[0]
    _check_out(h, (slots, C), torch.float32, "h", what)
    there = _elsewhere(x, stream)
    if there is not None:
        with there:
            return gated_scan_step(x, r, i, decay, h, index=index, out=out)
    stream = _raw_stream(x.get_device())
    decay = _decay(decay, C, what)
    fill = out is None
    if fill:
        out = _new_like(x)
    else:
        _check_out(out, x.shape, x.dtype, "out", what)
    x, _, xt = _rows(x, True)
    r, _, rt = _rows(r, True)
    i, _, it = _rows(i, True)
    _raise(_lib()["gated_scan_step"](x.data_ptr(), r.data_ptr(), i.data_ptr(), decay.data_ptr(), h.data_ptr(),
                                     _ptr(index), out.data_ptr(), B, slots, C, xt, rt, it, fill, code, stream),
           what)
    return out
