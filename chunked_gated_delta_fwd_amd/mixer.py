"""The operators around the recurrence in a token mixer, on torch tensors in
device memory: the short causal convolution, the query/key norm with the
position rotation, and the selective state space scan.

Marshalling only, as in the package's other calls: every value is computed by
the kernels behind ``include/gdr.h``, which documents shapes, dtypes and
errors.  These calls are made once per layer and token while decoding, where
building descriptor objects would take longer than the kernel, so the
descriptors of a call are packed into one buffer per thread (the library reads
them before it returns).
"""
from __future__ import annotations

import ctypes
import struct
import threading

import torch

from . import GDR_BF16, GDR_F32, GDR_I32, GdrError, _check, library

ACTIVATIONS = {None: 0, "none": 0, "silu": 1, "swish": 1}
NORMS = {"l2": 0, "rms": 1}

_CODE = {torch.float32: GDR_F32, torch.bfloat16: GDR_BF16, torch.int32: GDR_I32}
_MAX_DIMS, _SLOTS = 5, 24
# a gdr_tensor followed by its shape and strides
_SLOT = 32 + 16 * _MAX_DIMS
_PACK = [struct.Struct("<QiiQQ%dq%dx%dq" % (n, 8 * (_MAX_DIMS - n), n)) for n in range(_MAX_DIMS + 1)]


class _Buffer(threading.local):
    def __init__(self):
        self.raw = ctypes.create_string_buffer(_SLOT * _SLOTS)
        base = ctypes.addressof(self.raw)
        self.at = [base + i * _SLOT for i in range(_SLOTS)]


_buffer = _Buffer()


def _call(entry, tensors, *rest):
    """entry(descriptor addresses of `tensors` (None: NULL), *rest, stream); raises on a status."""
    buf = _buffer
    raw, at = buf.raw, buf.at
    args = []
    dev = tensors[0].get_device()
    for i, t in enumerate(tensors):
        if t is None:
            args.append(None)
            continue
        code = _CODE.get(t.dtype)
        if code is None:
            raise GdrError(-3, "unsupported dtype %s" % t.dtype)
        if t.get_device() != dev or dev < 0:
            raise GdrError(-6, "every tensor has to be on one GPU (argument %d is on %s)" % (i, t.device))
        n = t.dim()
        if n > _MAX_DIMS:
            raise GdrError(-2, "argument %d has %d dimensions" % (i, n))
        a = at[i]
        _PACK[n].pack_into(raw, i * _SLOT, t.data_ptr(), code, n, a + 32, a + 32 + 8 * _MAX_DIMS, *t.shape, *t.stride())
        args.append(a)
    if dev != torch.cuda.current_device():
        with torch.cuda.device(dev):
            status = entry(*args, *rest, torch.cuda.current_stream(dev).cuda_stream)
    else:
        status = entry(*args, *rest, torch.cuda.current_stream(dev).cuda_stream)
    if status:
        _check(library(), status)


def _call_ws(entry, tensors, *rest):
    """_call for an entry with a workspace: the library's own, or in a stream
    capture one from torch's allocator, which belongs to the graph then."""
    if not torch.cuda.is_current_stream_capturing():
        return _call(entry, tensors, *rest, None, None)
    size = ctypes.c_int64(0)
    _call(entry, tensors, *rest, None, ctypes.addressof(size))
    ws = torch.empty(max(size.value, 16), dtype=torch.uint8, device=tensors[0].device)
    size.value = ws.numel()
    _call(entry, tensors, *rest, ws.data_ptr(), ctypes.addressof(size))


def _choice(table, value, what):
    if value not in table:
        raise GdrError(-1, "%s: %r is none of %s" % (what, value, sorted(str(k) for k in table)))
    return table[value]


def _n_seq(x, cu_seqlens):
    return x.shape[0] if cu_seqlens is None else cu_seqlens.shape[0] - 1


def short_conv_fwd(x, w, bias=None, cu_seqlens=None, s0=None, activation="silu", output_final_state=True, y=None, st=None):
    """Short causal depthwise convolution: x ``[B, T, ch]`` (rows may be a slice
    of a wider projection), w ``[ch, W]`` with W = 2, 3 or 4, bias ``[ch]``,
    ``cu_seqlens`` int32 ``[N+1]`` (B == 1), state s0 ``[N, W-1, ch]`` or None
    for zeros, activation ``"silu"`` or None.  Returns ``(y, st)``: st
    ``[N, W-1, ch]`` is the state after the call (None unless
    ``output_final_state``); a length-0 sequence hands its s0 on."""
    act = _choice(ACTIVATIONS, activation, "activation")
    if y is None:
        y = x.new_empty(x.shape)
    if st is None and output_final_state:
        st = x.new_empty((_n_seq(x, cu_seqlens), w.shape[1] - 1, x.shape[-1]))
    _call(library().gdr_short_conv_fwd, (x, w, bias, cu_seqlens, s0, y, st), act)
    return y, st


def short_conv_bwd(x, w, dy, bias=None, cu_seqlens=None, s0=None, dst=None, activation="silu",
                   dx=None, dw=None, db=None, ds0=None, want_ds0=True):
    """Gradients of ``short_conv_fwd`` given dy ``[B, T, ch]`` and dst (gradient
    of st, or None): ``(dx, dw, db, ds0)``, dx and ds0 in x's dtype, dw
    ``[ch, W]`` and db ``[ch]`` fp32 (db None without bias)."""
    act = _choice(ACTIVATIONS, activation, "activation")
    if dx is None:
        dx = x.new_empty(x.shape)
    if dw is None:
        dw = x.new_empty(w.shape, dtype=torch.float32)
    if db is None and bias is not None:
        db = x.new_empty(bias.shape, dtype=torch.float32)
    if ds0 is None and want_ds0:
        ds0 = x.new_empty((_n_seq(x, cu_seqlens), w.shape[1] - 1, x.shape[-1]))
    _call_ws(library().gdr_short_conv_bwd, (x, w, bias, cu_seqlens, s0, dy, dst, dx, dw, db, ds0), act)
    return dx, dw, db, ds0


def short_conv_step(x, state, w, bias=None, activation="silu", y=None):
    """One token per sequence: x ``[B, ch]``, state ``[B, W-1, ch]`` updated in
    place.  Returns y ``[B, ch]``."""
    act = _choice(ACTIVATIONS, activation, "activation")
    if y is None:
        y = x.new_empty(x.shape)
    _call(library().gdr_short_conv_step, (x, state, w, bias, y), act)
    return y


def qk_norm_rope_fwd(q, k, wq=None, wk=None, cos=None, sin=None, positions=None, norm="rms", eps=1e-6,
                     interleaved=False, oq=None, ok=None):
    """Norm (``"rms"`` or ``"l2"``) of every head of q ``[B, T, Hq, d]`` and k
    ``[B, T, Hk, d]`` with weights ``[d]`` or None, then, with fp32 tables cos
    and sin ``[table, rot / 2]``, the rotation of the first rot channels at
    positions int32 ``[B, T]`` (None: 0 .. T-1).  Returns ``(oq, ok)``."""
    kind = _choice(NORMS, norm, "norm")
    if oq is None:
        oq = q.new_empty(q.shape)
    if ok is None:
        ok = k.new_empty(k.shape)
    _call(library().gdr_qk_norm_rope_fwd, (q, k, wq, wk, cos, sin, positions, oq, ok), kind, eps, int(interleaved))
    return oq, ok


def qk_norm_rope_bwd(q, k, doq, dok, wq=None, wk=None, cos=None, sin=None, positions=None, norm="rms", eps=1e-6,
                     interleaved=False, dq=None, dk=None, dwq=None, dwk=None):
    """Gradients of ``qk_norm_rope_fwd``: ``(dq, dk, dwq, dwk)``, dwq and dwk
    fp32 ``[d]`` (None without the weight)."""
    kind = _choice(NORMS, norm, "norm")
    if dq is None:
        dq = q.new_empty(q.shape)
    if dk is None:
        dk = k.new_empty(k.shape)
    if dwq is None and wq is not None:
        dwq = q.new_empty(wq.shape, dtype=torch.float32)
    if dwk is None and wk is not None:
        dwk = k.new_empty(wk.shape, dtype=torch.float32)
    _call_ws(library().gdr_qk_norm_rope_bwd, (q, k, wq, wk, cos, sin, positions, doq, dok, dq, dk, dwq, dwk), kind, eps,
             int(interleaved))
    return dq, dk, dwq, dwk


def ssm_scan_fwd(x, dt, A, b, c, D=None, dt_bias=None, cu_seqlens=None, h0=None, output_final_state=True, y=None, ht=None):
    """Selective state space scan: x ``[B, T, H, p]``, raw dt ``[B, T, H]``, A
    ``[H]``, b and c ``[B, T, G, n]``, D and dt_bias ``[H]`` or None,
    ``cu_seqlens`` int32 ``[N+1]`` (B == 1), h0 fp32 ``[N, H, n, p]`` or None.
    Returns ``(y, ht)``; ht is None unless ``output_final_state``, and a
    length-0 sequence hands its h0 on."""
    if y is None:
        y = x.new_empty(x.shape)
    if ht is None and output_final_state:
        ht = x.new_empty((_n_seq(x, cu_seqlens), x.shape[2], b.shape[3], x.shape[3]), dtype=torch.float32)
    _call_ws(library().gdr_ssm_scan_fwd, (x, dt, A, b, c, D, dt_bias, cu_seqlens, h0, y, ht))
    return y, ht


def ssm_scan_bwd(x, dt, A, b, c, dy, D=None, dt_bias=None, cu_seqlens=None, h0=None, dht=None, want_dh0=True,
                 dx=None, ddt=None, dA=None, db=None, dc=None, dD=None, ddt_bias=None, dh0=None):
    """Gradients of ``ssm_scan_fwd`` given dy ``[B, T, H, p]`` and dht (gradient
    of ht, or None): ``(dx, ddt, dA, db, dc, dD, ddt_bias, dh0)`` in the dtypes
    of their inputs (dD and ddt_bias None without the input, dh0 None when
    ``want_dh0`` is False)."""
    if dx is None:
        dx = x.new_empty(x.shape)
    if ddt is None:
        ddt = dt.new_empty(dt.shape)
    if dA is None:
        dA = A.new_empty(A.shape)
    if db is None:
        db = b.new_empty(b.shape)
    if dc is None:
        dc = c.new_empty(c.shape)
    if dD is None and D is not None:
        dD = A.new_empty(A.shape)
    if ddt_bias is None and dt_bias is not None:
        ddt_bias = A.new_empty(A.shape)
    if dh0 is None and want_dh0:
        dh0 = x.new_empty((_n_seq(x, cu_seqlens), x.shape[2], b.shape[3], x.shape[3]), dtype=torch.float32)
    _call_ws(library().gdr_ssm_scan_bwd,
             (x, dt, A, b, c, D, dt_bias, cu_seqlens, h0, dy, dht, dx, ddt, dA, db, dc, dD, ddt_bias, dh0))
    return dx, ddt, dA, db, dc, dD, ddt_bias, dh0


def ssm_step(x, dt, A, b, c, h, D=None, dt_bias=None, y=None):
    """One token of the state space scan per sequence: x ``[B, H, p]``, dt
    ``[B, H]``, A ``[H]``, b and c ``[B, G, n]``, state h fp32 ``[B, H, n, p]``
    updated in place.  Returns y ``[B, H, p]``."""
    if y is None:
        y = x.new_empty(x.shape)
    _call(library().gdr_ssm_step, (x, dt, A, b, c, D, dt_bias, h, y))
    return y
