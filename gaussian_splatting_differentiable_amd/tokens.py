"""Token operators: attention, the norm and rotation of queries and keys, dropout.

For models that predict Gaussians from the tokens of image patches and train
through the rasterizer. The work runs in the HIP kernels behind the calls that
``include/gs.h`` declares under "token operators"; the functions here check
shapes, allocate outputs and workspaces, and enqueue on the current stream (or
``stream``). They do no arithmetic of their own.

Tensors are ``[batch, tokens, heads, dim]`` with any strides whose innermost is 1
(views of a joint projection, say). The ``*_bwd`` functions take and return
gradients explicitly; ``Attention``, ``QkNormRope`` and ``Dropout`` are the same
calls for autograd.
"""
from __future__ import annotations

import contextlib
import ctypes as C
import functools
import math
from struct import Struct

import torch

from . import GS_OK, GsError, lib

F32, BF16, F16 = 0, 1, 2
_DTYPES = {torch.float32: F32, torch.bfloat16: BF16, torch.float16: F16}


# gs_tokens, gs_qk_shape and gs_attn_shape of include/gs.h as bytes, which ctypes passes
# by address: building a Structure for every tensor costs more than a small call's kernel.
_TOKENS, _QK, _ATTN = Struct("=4q"), Struct("=9ifq"), Struct("=8if4xq")


def _declare(L):
    P, sz, i32, i64 = C.c_void_p, C.c_size_t, C.c_int32, C.c_int64
    T = Q = A = C.c_char_p
    L.gs_qk_workspace_size.argtypes, L.gs_qk_workspace_size.restype = [Q], sz
    L.gs_attention_workspace_size.argtypes, L.gs_attention_workspace_size.restype = [A], sz
    L.gs_attention_bwd_workspace_size.argtypes = [A]
    L.gs_attention_bwd_workspace_size.restype = sz
    L.gs_qk_norm_rope.argtypes = [Q, T, T, P, P, P, P, T, T, P]
    L.gs_qk_norm_rope_bwd.argtypes = [Q, T, T, T, T, P, P, P, P, T, T, P, P, P, sz, P]
    L.gs_attention.argtypes = [A, T, T, T, P, T, P, P, sz, P]
    L.gs_attention_bwd.argtypes = [A, T, T, T, T, P, T, P, T, T, T, P, sz, P]
    L.gs_dropout.argtypes = [i64, i64, i32, P, i64, P, i64, P, i64, C.c_double, C.c_uint64,
                             C.c_uint64, i32, P]
    for name in ("gs_qk_norm_rope", "gs_qk_norm_rope_bwd", "gs_attention", "gs_attention_bwd",
                 "gs_dropout"):
        getattr(L, name).restype = i32


_declared = None


def _lib():
    global _declared
    L = lib()
    if _declared is not L:
        _declare(L)
        _declared = L
    return L


def _check(status, what):
    if status != GS_OK:
        raise GsError(status, what)


def _tokens(t):
    """The C view of a [batch, tokens, heads, dim] tensor (None: absent)."""
    if t is None:
        return None
    s = t.stride()
    return _TOKENS.pack(t.data_ptr(), s[0], s[1], s[2])


def _same(name, t, shape, dtype, device):
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype} on {device}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")
    _inner(name, t)


def _inner(name, t):
    if t.stride(-1) != 1 and t.dim() == 4 and t.shape[3] != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")


def _base(name, t):
    if not t.is_cuda:
        raise ValueError(f"{name}: expected a device tensor")
    if t.dim() != 4:
        raise ValueError(f"{name}: expected [batch, tokens, heads, dim]")
    if t.dtype not in _DTYPES:
        raise ValueError(f"{name}: unsupported type {t.dtype}")
    _inner(name, t)


_HERE = contextlib.nullcontext()


def _on(stream, *tensors):
    """The context calls allocate and launch in: the tensors' device and `stream`, on which
    the tensors are then marked as used."""
    if stream is None:
        device = tensors[0].device
        return _HERE if device.index == torch.cuda.current_device() else torch.cuda.device(device)
    for t in tensors:
        if t is not None:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def _stream(stream, device):
    """The handle of `stream`, or of the device's current stream."""
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(device.index)


def _addr(t):
    return None if t is None else t.data_ptr()


def _list2d(name, t, batch, n, tail, device):
    """(pointer, entries from one batch entry to the next) of an int32 list that is one per
    batch entry or shared by all."""
    if t is None:
        return None, 0
    if t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous int32 tensor on {device}")
    if t.shape == (n, *tail):
        return t.data_ptr(), 0
    if t.shape == (batch, n, *tail):
        return t.data_ptr(), n
    raise ValueError(f"{name}: expected {(n, *tail)} or {(batch, n, *tail)}, got {tuple(t.shape)}")


def _vector(name, t, n, device):
    if t is None:
        return None
    if t.shape != (n,) or t.dtype != torch.float32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected {n} contiguous float32 values on {device}")
    return t.data_ptr()


# ------------------------------------------------------------------ norm and rotation

def _qk_shape(q, k, cos_sin, positions, neighbours, eps):
    x = q if q is not None else k
    if x is None:
        raise ValueError("queries or keys are needed")
    _base("q" if q is not None else "k", x)
    B, n, _, d = x.shape
    if q is not None and k is not None:
        _same("k", k, (B, n, k.shape[2], d), q.dtype, q.device)
    rot = rows = 0
    if cos_sin is not None:
        if cos_sin.dim() != 2 or cos_sin.dtype != torch.float32 or cos_sin.device != x.device \
                or not cos_sin.is_contiguous():
            raise ValueError("cos_sin: expected contiguous [positions, rot_dim] float32 on the "
                             "same device")
        rows, rot = cos_sin.shape
    pos, stride = _list2d("positions", positions, B, n, (), x.device)
    shape = _QK.pack(B, n, 0 if q is None else q.shape[2], 0 if k is None else k.shape[2], d,
                     _DTYPES[x.dtype], rot, bool(neighbours), rows, eps, stride)
    return shape, x, pos


def _like(t, out=None, name="out"):
    if t is None:
        return None
    if out is None:
        return torch.empty(t.shape, dtype=t.dtype, device=t.device)
    _same(name, out, t.shape, t.dtype, t.device)
    return out


def qk_norm_rope(q, k, q_weight=None, k_weight=None, *, cos_sin=None, positions=None,
                 neighbours=False, eps=1e-6, q_out=None, k_out=None, stream=None):
    """The norm of each head's queries and keys and the rotation by position, in one pass.

    q, k: [batch, tokens, heads, dim] (either may be None); weights [dim] float32 or None;
    cos_sin [positions, rot_dim] float32: cosines, then sines (None: no rotation); positions
    [batch, tokens] or [tokens] int32 rows of it (None: row t for token t). q_out, k_out may be
    the inputs. Returns (q_out, k_out)."""
    shape, x, pos = _qk_shape(q, k, cos_sin, positions, neighbours, eps)
    wq = _vector("q_weight", q_weight, x.shape[3], x.device)
    wk = _vector("k_weight", k_weight, x.shape[3], x.device)
    with _on(stream, x, q, k, q_weight, k_weight, cos_sin, positions):
        q_out, k_out = _like(q, q_out, "q_out"), _like(k, k_out, "k_out")
        _check(_lib().gs_qk_norm_rope(shape, _tokens(q), _tokens(k), wq, wk, _addr(cos_sin), pos,
                                      _tokens(q_out), _tokens(k_out), _stream(stream, x.device)),
               "gs_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, *, cos_sin=None,
                     positions=None, neighbours=False, eps=1e-6, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) from those of qk_norm_rope's outputs; None for
    what was None."""
    shape, x, pos = _qk_shape(q, k, cos_sin, positions, neighbours, eps)
    d, dev = x.shape[3], x.device
    for name, g, t in (("dq_out", dq_out, q), ("dk_out", dk_out, k)):
        if t is not None:
            _same(name, g, t.shape, t.dtype, dev)
    wq, wk = _vector("q_weight", q_weight, d, dev), _vector("k_weight", k_weight, d, dev)
    L = _lib()
    with _on(stream, x, q, k, dq_out, dk_out, q_weight, k_weight, cos_sin, positions):
        dq, dk = _like(q), _like(k)
        dwq, dwk = (None if w is None else torch.empty(d, dtype=torch.float32, device=dev)
                    for w in (q_weight, k_weight))
        ws, size = None, 0
        if dwq is not None or dwk is not None:
            size = L.gs_qk_workspace_size(shape)
            ws = torch.empty(size, dtype=torch.uint8, device=dev)
        _check(L.gs_qk_norm_rope_bwd(shape, _tokens(dq_out if q is not None else None),
                                     _tokens(dk_out if k is not None else None), _tokens(q),
                                     _tokens(k), wq, wk, _addr(cos_sin), pos, _tokens(dq),
                                     _tokens(dk), _addr(dwq), _addr(dwk), _addr(ws), size,
                                     _stream(stream, dev)),
               "gs_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


# ------------------------------------------------------------------ attention

def _attn_shape(q, k, v, spans, causal, scale):
    _base("q", q)
    _base("k", k)
    B, n, H, d = q.shape
    _same("k", k, (B, k.shape[1], k.shape[2], d), q.dtype, q.device)
    _same("v", v, k.shape, q.dtype, q.device)
    at, stride = _list2d("spans", spans, B, n, (2,), q.device)
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    return _ATTN.pack(B, H, k.shape[2], n, k.shape[1], d, _DTYPES[q.dtype], bool(causal), scale,
                      stride), at


def attention_workspace_size(q, k, *, causal=False, backward=False) -> int:
    """Bytes of workspace an attention (or its backward) of these sizes takes."""
    shape, _ = _attn_shape(q, k, k, None, causal, None)
    return _attn_bytes(shape, backward)


@functools.lru_cache(maxsize=256)
def _attn_bytes(shape, backward):
    L = _lib()
    return (L.gs_attention_bwd_workspace_size if backward else L.gs_attention_workspace_size)(shape)


def _workspace(size, given, device):
    if given is None:
        return torch.empty(size, dtype=torch.uint8, device=device) if size else None
    if given.numel() * given.element_size() < size:
        raise ValueError(f"workspace: {size} bytes are needed")
    return given


def attention(q, k, v, *, spans=None, causal=False, scale=None, out=None, workspace=None,
              stream=None):
    """softmax(scale q k^T) v over the keys each query sees; returns (o, lse).

    q [batch, q_tokens, q_heads, dim], k and v [batch, kv_tokens, kv_heads, dim], bfloat16 or
    float16; scale 1 / sqrt(dim) by default; spans [q_tokens, 2] or [batch, q_tokens, 2] int32:
    each query's keys [lo, hi); causal: query t sees keys up to t + kv_tokens - q_tokens. A
    query that sees no key gets 0 and lse = -inf. lse is [batch, q_heads, q_tokens] float32."""
    shape, at = _attn_shape(q, k, v, spans, causal, scale)
    L = _lib()
    with _on(stream, q, k, v, spans):
        o = _like(q, out)
        lse = torch.empty((q.shape[0], q.shape[2], q.shape[1]), dtype=torch.float32,
                          device=q.device)
        size = _attn_bytes(shape, False)
        ws = _workspace(size, workspace, q.device)
        _check(L.gs_attention(shape, _tokens(q), _tokens(k), _tokens(v), at, _tokens(o), _addr(lse),
                              _addr(ws), size, _stream(stream, q.device)),
               "gs_attention")
    return o, lse


def attention_bwd(do, q, k, v, o, lse, *, spans=None, causal=False, scale=None, workspace=None,
                  stream=None):
    """Gradients (dq, dk, dv) of attention from that of o, with its o and lse."""
    shape, at = _attn_shape(q, k, v, spans, causal, scale)
    _same("do", do, q.shape, q.dtype, q.device)
    _same("o", o, q.shape, q.dtype, q.device)
    _same("lse", lse, (q.shape[0], q.shape[2], q.shape[1]), torch.float32, q.device)
    L = _lib()
    with _on(stream, q, k, v, spans, do, o, lse):
        dq, dk, dv = _like(q), _like(k), _like(k)
        size = _attn_bytes(shape, True)
        ws = _workspace(size, workspace, q.device)
        _check(L.gs_attention_bwd(shape, _tokens(do), _tokens(q), _tokens(k), _tokens(v), at,
                                  _tokens(o), _addr(lse), _tokens(dq), _tokens(dk), _tokens(dv),
                                  _addr(ws), size, _stream(stream, q.device)),
               "gs_attention_bwd")
    return dq, dk, dv


# ------------------------------------------------------------------ dropout

def _row_stride(name, t, rows, cols):
    """Elements from one row to the next of t seen as [rows][cols]."""
    if t.is_contiguous():
        return cols
    if t.dim() == 2 and (t.stride(1) == 1 or cols == 1):
        return t.stride(0)
    if t.dim() == 1:
        return t.stride(0)
    raise ValueError(f"{name}: expected a contiguous tensor, or rows that are contiguous")


def dropout(x, p, seed, offset=0, *, residual=None, per_row=False, out=None, stream=None):
    """residual + keep x / (1 - p), keep from the counter-based generator (seed, offset).

    per_row: one draw for each row (the last dimension) instead of each element. The gradient
    with respect to x is dropout(dy, p, seed, offset, per_row=...). A call takes
    ceil(draws / 4) counters from `offset` on."""
    if not x.is_cuda or x.dtype not in _DTYPES:
        raise ValueError("x: expected a float32, bfloat16 or float16 device tensor")
    if x.dim() > 1:
        cols = x.shape[-1]
        rows = x.numel() // cols if cols else 0
    elif per_row:
        raise ValueError("per_row takes at least two dimensions")
    else:
        rows, cols = x.numel(), 1
    dev = x.device
    with _on(stream, x, residual):
        if out is None:
            out = torch.empty(x.shape, dtype=x.dtype, device=dev)
        else:
            _same("out", out, x.shape, x.dtype, dev)
        if residual is not None:
            _same("residual", residual, x.shape, x.dtype, dev)
        _check(_lib().gs_dropout(
            rows, cols, _DTYPES[x.dtype], x.data_ptr(), _row_stride("x", x, rows, cols),
            _addr(residual),
            0 if residual is None else _row_stride("residual", residual, rows, cols),
            out.data_ptr(), _row_stride("out", out, rows, cols), p, seed & (2 ** 64 - 1),
            offset & (2 ** 64 - 1), bool(per_row), _stream(stream, dev)), "gs_dropout")
    return out


# ------------------------------------------------------------------ autograd

class QkNormRope(torch.autograd.Function):
    """QkNormRope.apply(q, k, q_weight, k_weight, cos_sin, positions, neighbours, eps)."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos_sin, positions, neighbours, eps):
        ctx.save_for_backward(q, k, q_weight, k_weight, cos_sin, positions)
        ctx.how = dict(neighbours=neighbours, eps=eps)
        return qk_norm_rope(q, k, q_weight, k_weight, cos_sin=cos_sin, positions=positions,
                            **ctx.how)

    @staticmethod
    def backward(ctx, dq, dk):
        q, k, q_weight, k_weight, cos_sin, positions = ctx.saved_tensors
        g = qk_norm_rope_bwd(dq.contiguous(), dk.contiguous(), q, k, q_weight, k_weight,
                             cos_sin=cos_sin, positions=positions, **ctx.how)
        return (*g, None, None, None, None)


class Attention(torch.autograd.Function):
    """Attention.apply(q, k, v, spans, causal, scale) -> o."""

    @staticmethod
    def forward(ctx, q, k, v, spans, causal, scale):
        o, lse = attention(q, k, v, spans=spans, causal=causal, scale=scale)
        ctx.save_for_backward(q, k, v, spans, o, lse)
        ctx.how = dict(causal=causal, scale=scale)
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, spans, o, lse = ctx.saved_tensors
        return (*attention_bwd(do.contiguous(), q, k, v, o, lse, spans=spans, **ctx.how),
                None, None, None)


class Dropout(torch.autograd.Function):
    """Dropout.apply(x, residual, p, seed, offset, per_row)."""

    @staticmethod
    def forward(ctx, x, residual, p, seed, offset, per_row):
        ctx.how = (p, seed, offset)
        ctx.per_row, ctx.residual = per_row, residual is not None
        return dropout(x, p, seed, offset, residual=residual, per_row=per_row)

    @staticmethod
    def backward(ctx, dy):
        dy = dy.contiguous()
        return (dropout(dy, *ctx.how, per_row=ctx.per_row), dy if ctx.residual else None,
                None, None, None, None)
