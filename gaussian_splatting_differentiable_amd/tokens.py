"""Token operators: attention, the norm and rotation of queries and keys, dropout.

For models that predict Gaussians from the tokens of image patches and train
through the rasterizer. The work runs in the HIP kernels behind the calls that
``include/gs.h`` declares under "token operators"; the functions here check
shapes, allocate outputs and workspaces, and enqueue on the current stream (or
``stream``). They do no arithmetic of their own.

Tensors are ``[batch, tokens, heads, dim]`` by their strides (views of a joint
projection, say): the elements of a head are contiguous, the tensor and its other
strides are multiples of 16 bytes, and tokens are less than 2^23 elements apart; what
does not fit is refused. The ``*_bwd`` functions take and return
gradients explicitly; ``Attention``, ``QkNormRope`` and ``Dropout`` are the same
calls for autograd (the first two have no second derivative: asking for it is an error).
"""
from __future__ import annotations

import contextlib
import ctypes as C
import functools
import math
from struct import Struct

import torch
from torch.autograd.function import once_differentiable

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
    """The C view of a [batch, tokens, heads, dim] tensor."""
    s = t.stride()
    if s[3] != 1 and t.shape[3] != 1:
        raise ValueError("the elements of a head must be contiguous")
    return _TOKENS.pack(t.data_ptr(), s[0], s[1], s[2])


def _same(name, t, shape, dtype, device):
    if t.shape != shape or t.dtype != dtype or t.device != device:
        raise ValueError(f"{name}: expected {tuple(shape)} {dtype} on {device}, got "
                         f"{tuple(t.shape)} {t.dtype} on {t.device}")


def _whole(name, t, shape, dtype, device):
    _same(name, t, shape, dtype, device)
    if not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous tensor")
    return t.data_ptr()


def _base(name, shape, dtype, device):
    if device.type != "cuda":
        raise ValueError(f"{name}: expected a device tensor")
    if len(shape) != 4:
        raise ValueError(f"{name}: expected [batch, tokens, heads, dim]")
    if dtype not in _DTYPES:
        raise ValueError(f"{name}: unsupported type {dtype}")


def _elsewhere(stream, device):
    """Whether a call is not for the current stream of the current device."""
    if stream is not None and stream.device != device:
        raise ValueError(f"a stream of {stream.device} for tensors on {device}")
    return stream is not None or device.index != torch._C._cuda_getDevice()


@contextlib.contextmanager
def _there(stream, device, tensors):
    """That stream and device, to allocate and launch in; the tensors are marked as used on it."""
    with torch.cuda.device(device):
        if stream is None:
            yield
            return
        for t in tensors:
            if t is not None:
                t.record_stream(stream)
        with torch.cuda.stream(stream):
            yield


def _stream(device):
    """The handle of the device's current stream."""
    return torch._C._cuda_getCurrentRawStream(device.index)


def _addr(t):
    return None if t is None else t.data_ptr()


def _list2d(name, t, batch, n, tail, device):
    """(pointer, entries from one batch entry to the next) of an int32 list that is one per
    batch entry or shared by all."""
    if t.dtype != torch.int32 or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name}: expected a contiguous int32 tensor on {device}")
    if t.shape == (n, *tail):
        return t.data_ptr(), 0
    if t.shape == (batch, n, *tail):
        return t.data_ptr(), n
    raise ValueError(f"{name}: expected {(n, *tail)} or {(batch, n, *tail)}, got {tuple(t.shape)}")


def _out(name, out, like):
    if out is None:
        return torch.empty_like(like, memory_format=torch.contiguous_format)
    _same(name, out, like.shape, like.dtype, like.device)
    torch.autograd.graph.increment_version(out)  # autograd sees that it is overwritten
    return out


# ------------------------------------------------------------------ norm and rotation

def _about(t):
    return None if t is None else (t.shape, t.dtype, t.device)


@functools.lru_cache(maxsize=256)
def _qk_plan(q, k, q_weight, k_weight, cos_sin, positions, neighbours, eps):
    """The C shape from the (shape, type, device) of the tensors, and the workspace."""
    if q is None and k is None:
        raise ValueError("queries or keys are needed")
    (B, n, _, d), dt, dev = _sized("q", q) if q is not None else _sized("k", k)
    if q is not None and k is not None:
        (kb, kn, _, kd), kt, kdev = _sized("k", k)
        if (kb, kn, kd, kt, kdev) != (B, n, d, dt, dev):
            raise ValueError(f"q {q} and k {k} do not fit")
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None and w != (torch.Size((d,)), torch.float32, dev):
            raise ValueError(f"{name}: expected {d} float32 values on {dev}")
    rot = rows = stride = 0
    if cos_sin is not None:
        if len(cos_sin[0]) != 2 or cos_sin[1:] != (torch.float32, dev):
            raise ValueError(f"cos_sin: expected [positions, rot_dim] float32 on {dev}")
        rows, rot = cos_sin[0]
    if positions is not None:
        if positions[0] not in ((n,), (B, n)) or positions[1:] != (torch.int32, dev):
            raise ValueError(f"positions: expected {(n,)} or {(B, n)} int32 on {dev}")
        stride = n if len(positions[0]) == 2 else 0
    shape = _QK.pack(B, n, 0 if q is None else q[0][2], 0 if k is None else k[0][2], d,
                     _DTYPES[dt], rot, neighbours, rows, eps, stride)
    return shape, _lib().gs_qk_workspace_size(shape)


def _sized(name, about):
    _base(name, *about)
    return about


def _qk_args(q, k, q_weight, k_weight, cos_sin, positions, neighbours, eps):
    """(shape, workspace bytes, q view, k view, weight, table and position pointers, device)
    after the checks."""
    shape, size = _qk_plan(_about(q), _about(k), _about(q_weight), _about(k_weight),
                           _about(cos_sin), _about(positions), bool(neighbours), float(eps))
    at = []
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight), ("cos_sin", cos_sin),
                    ("positions", positions)):
        if t is not None and not t.is_contiguous():
            raise ValueError(f"{name}: expected a contiguous tensor")
        at.append(None if t is None else t.data_ptr())
    return (shape, size, None if q is None else _tokens(q), None if k is None else _tokens(k), at,
            (q if q is not None else k).device)


def qk_norm_rope(q, k, q_weight=None, k_weight=None, *, cos_sin=None, positions=None,
                 neighbours=False, eps=1e-6, q_out=None, k_out=None, stream=None):
    """The norm of each head's queries and keys and the rotation by position, in one pass.

    q, k: [batch, tokens, heads, dim] (either may be None); weights [dim] float32 or None;
    cos_sin [positions, rot_dim] float32: cosines, then sines (None: no rotation); positions
    [batch, tokens] or [tokens] int32 rows of it (None: row t for token t). q_out, k_out may be
    the inputs. Returns (q_out, k_out)."""
    shape, size, tq, tk, at, dev = _qk_args(q, k, q_weight, k_weight, cos_sin, positions,
                                            neighbours, eps)
    if _elsewhere(stream, dev):
        with _there(stream, dev, (q, k, q_weight, k_weight, cos_sin, positions, q_out, k_out)):
            return qk_norm_rope(q, k, q_weight, k_weight, cos_sin=cos_sin, positions=positions,
                                neighbours=neighbours, eps=eps, q_out=q_out, k_out=k_out)
    q_out = None if q is None else _out("q_out", q_out, q)
    k_out = None if k is None else _out("k_out", k_out, k)
    _check(_lib().gs_qk_norm_rope(shape, tq, tk, *at,
                                  None if q is None else _tokens(q_out),
                                  None if k is None else _tokens(k_out), _stream(dev)),
           "gs_qk_norm_rope")
    return q_out, k_out


def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, *, cos_sin=None,
                     positions=None, neighbours=False, eps=1e-6, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) from those of qk_norm_rope's outputs; None for
    what was None."""
    shape, size, tq, tk, at, dev = _qk_args(q, k, q_weight, k_weight, cos_sin, positions,
                                            neighbours, eps)
    if _elsewhere(stream, dev):
        with _there(stream, dev, (dq_out, dk_out, q, k, q_weight, k_weight, cos_sin, positions)):
            return qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight, k_weight, cos_sin=cos_sin,
                                    positions=positions, neighbours=neighbours, eps=eps)
    dq = dk = gq = gk = oq = ok = dwq = dwk = ws = None
    if q is not None:
        _same("dq_out", dq_out, q.shape, q.dtype, dev)
        dq = _out("dq", None, q)
        gq, oq = _tokens(dq_out), _tokens(dq)
    if k is not None:
        _same("dk_out", dk_out, k.shape, k.dtype, dev)
        dk = _out("dk", None, k)
        gk, ok = _tokens(dk_out), _tokens(dk)
    if q_weight is not None:
        dwq = _out("dq_weight", None, q_weight)
    if k_weight is not None:
        dwk = _out("dk_weight", None, k_weight)
    L = _lib()
    if dwq is not None or dwk is not None:
        ws = torch.empty(size, dtype=torch.uint8, device=dev)
    _check(L.gs_qk_norm_rope_bwd(shape, gq, gk, tq, tk, *at, oq, ok, _addr(dwq), _addr(dwk),
                                 _addr(ws), size, _stream(dev)),
           "gs_qk_norm_rope_bwd")
    return dq, dk, dwq, dwk


# ------------------------------------------------------------------ attention

@functools.lru_cache(maxsize=256)
def _attn_plan(qs, ks, vs, types, devices, causal, scale, stride):
    """What follows from the sizes: the C shape, that of the log sums, and the workspaces."""
    _base("q", qs, types[0], devices[0])
    _base("k", ks, types[1], devices[1])
    B, n, H, d = qs
    if ks[0] != B or ks[3] != d or vs != ks or len(set(types)) > 1 or len(set(devices)) > 1:
        raise ValueError(f"q {tuple(qs)} {types[0]} on {devices[0]}, k {tuple(ks)} {types[1]} on "
                         f"{devices[1]}, v {tuple(vs)} {types[2]} on {devices[2]} do not fit")
    if scale is None:
        scale = 1.0 / math.sqrt(d)
    shape = _ATTN.pack(B, H, ks[2], n, ks[1], d, _DTYPES[types[0]], causal, scale, stride)
    L = _lib()
    return (shape, (B, H, n), L.gs_attention_workspace_size(shape),
            L.gs_attention_bwd_workspace_size(shape))


def _attn_args(q, k, v, spans, causal, scale):
    at, stride = None, 0
    if spans is not None:
        if q.dim() != 4:
            raise ValueError("q: expected [batch, tokens, heads, dim]")
        at, stride = _list2d("spans", spans, q.shape[0], q.shape[1], (2,), q.device)
    return at, _attn_plan(q.shape, k.shape, v.shape, (q.dtype, k.dtype, v.dtype),
                          (q.device, k.device, v.device), bool(causal),
                          None if scale is None else float(scale), stride)


def attention_workspace_size(q, k, *, causal=False, backward=False) -> int:
    """Bytes of workspace an attention (or its backward) of these sizes takes."""
    _, plan = _attn_args(q, k, k, None, causal, None)
    return plan[3 if backward else 2]


def _workspace(size, given, device):
    if given is None:
        return torch.empty(size, dtype=torch.uint8, device=device) if size else None
    if given.device != device or not given.is_contiguous() or \
            given.numel() * given.element_size() < size:
        raise ValueError(f"workspace: {size} contiguous bytes on {device} are needed")
    return given


def attention(q, k, v, *, spans=None, causal=False, scale=None, out=None, workspace=None,
              stream=None):
    """softmax(scale q k^T) v over the keys each query sees; returns (o, lse).

    q [batch, q_tokens, q_heads, dim], k and v [batch, kv_tokens, kv_heads, dim], bfloat16 or
    float16; scale 1 / sqrt(dim) by default; spans [q_tokens, 2] or [batch, q_tokens, 2] int32:
    each query's keys [lo, hi); causal: query t sees keys up to t + kv_tokens - q_tokens. A
    query that sees no key gets 0 and lse = -inf. lse is [batch, q_heads, q_tokens] float32."""
    at, (shape, rows, size, _) = _attn_args(q, k, v, spans, causal, scale)
    dev = q.device
    if _elsewhere(stream, dev):
        with _there(stream, dev, (q, k, v, spans, out, workspace)):
            return attention(q, k, v, spans=spans, causal=causal, scale=scale, out=out,
                             workspace=workspace)
    o = _out("out", out, q)
    lse = torch.empty(rows, dtype=torch.float32, device=dev)
    ws = _workspace(size, workspace, dev) if size else None
    _check(_lib().gs_attention(shape, _tokens(q), _tokens(k), _tokens(v), at, _tokens(o),
                               lse.data_ptr(), _addr(ws), size, _stream(dev)),
           "gs_attention")
    return o, lse


def attention_bwd(do, q, k, v, o, lse, *, spans=None, causal=False, scale=None, workspace=None,
                  stream=None):
    """Gradients (dq, dk, dv) of attention from that of o, with its o and lse."""
    at, (shape, rows, _, size) = _attn_args(q, k, v, spans, causal, scale)
    dev = q.device
    _same("do", do, q.shape, q.dtype, dev)
    _same("o", o, q.shape, q.dtype, dev)
    sums = _whole("lse", lse, rows, torch.float32, dev)
    if _elsewhere(stream, dev):
        with _there(stream, dev, (do, q, k, v, o, lse, spans, workspace)):
            return attention_bwd(do, q, k, v, o, lse, spans=spans, causal=causal, scale=scale,
                                 workspace=workspace)
    dq = _out("dq", None, q)
    dk = _out("dk", None, k)
    dv = _out("dv", None, v)
    ws = _workspace(size, workspace, dev)
    _check(_lib().gs_attention_bwd(shape, _tokens(do), _tokens(q), _tokens(k), _tokens(v), at,
                                   _tokens(o), sums, _tokens(dq), _tokens(dk), _tokens(dv),
                                   _addr(ws), size, _stream(dev)),
           "gs_attention_bwd")
    return dq, dk, dv


# ------------------------------------------------------------------ dropout

def _row_stride(name, t, cols):
    """Elements from one row to the next of t seen as rows of `cols`."""
    if t.is_contiguous():
        return cols
    if t.dim() == 1 or (t.dim() == 2 and (t.stride(1) == 1 or cols == 1)):
        return t.stride(0)
    raise ValueError(f"{name}: expected a contiguous tensor, or rows that are contiguous")


def dropout(x, p, seed, offset=0, *, residual=None, per_row=False, out=None, stream=None):
    """residual + keep x / (1 - p), keep from the counter-based generator (seed, offset).

    per_row: one draw for each row (the last dimension) instead of each element. The gradient
    with respect to x is dropout(dy, p, seed, offset, per_row=...). A call takes
    ceil(draws / 4) counters from `offset` on."""
    dev = x.device
    if dev.type != "cuda" or x.dtype not in _DTYPES:
        raise ValueError("x: expected a float32, bfloat16 or float16 device tensor")
    if _elsewhere(stream, dev):
        with _there(stream, dev, (x, residual, out)):
            return dropout(x, p, seed, offset, residual=residual, per_row=per_row, out=out)
    if x.dim() > 1:
        cols = x.shape[-1]
        rows = x.numel() // cols if cols else 0
    elif per_row:
        raise ValueError("per_row takes at least two dimensions")
    else:
        rows, cols = x.numel(), 1
    out = _out("out", out, x)
    if residual is not None:
        _same("residual", residual, x.shape, x.dtype, dev)
    _check(_lib().gs_dropout(
        rows, cols, _DTYPES[x.dtype], x.data_ptr(), _row_stride("x", x, cols), _addr(residual),
        0 if residual is None else _row_stride("residual", residual, cols), out.data_ptr(),
        _row_stride("out", out, cols), p, seed & (2 ** 64 - 1), offset & (2 ** 64 - 1),
        bool(per_row), _stream(dev)), "gs_dropout")
    return out


# ------------------------------------------------------------------ autograd

def _no_gradient(ctx, **at):
    """Refuses a backward for arguments (name: place) that want a gradient and would get none."""
    for name, i in at.items():
        if ctx.needs_input_grad[i]:
            raise ValueError(f"{name}: no gradient is computed for it (detach it)")


class QkNormRope(torch.autograd.Function):
    """QkNormRope.apply(q, k, q_weight, k_weight, cos_sin, positions, neighbours, eps)."""

    @staticmethod
    def forward(ctx, q, k, q_weight, k_weight, cos_sin, positions, neighbours, eps):
        ctx.save_for_backward(q, k, q_weight, k_weight, cos_sin, positions)
        ctx.how = dict(neighbours=neighbours, eps=float(eps))  # as it is now
        return qk_norm_rope(q, k, q_weight, k_weight, cos_sin=cos_sin, positions=positions,
                            **ctx.how)

    @staticmethod
    @once_differentiable
    def backward(ctx, dq, dk):
        _no_gradient(ctx, cos_sin=4, eps=7)
        q, k, q_weight, k_weight, cos_sin, positions = ctx.saved_tensors
        dq, dk = (None if g is None else g.contiguous() for g in (dq, dk))  # None: was None
        g = qk_norm_rope_bwd(dq, dk, q, k, q_weight, k_weight, cos_sin=cos_sin,
                             positions=positions, **ctx.how)
        return (*g, None, None, None, None)


class Attention(torch.autograd.Function):
    """Attention.apply(q, k, v, spans, causal, scale) -> o."""

    @staticmethod
    def forward(ctx, q, k, v, spans, causal, scale):
        ctx.how = dict(causal=causal, scale=None if scale is None else float(scale))  # as it is now
        o, lse = attention(q, k, v, spans=spans, **ctx.how)
        ctx.save_for_backward(q, k, v, spans, o, lse)
        return o

    @staticmethod
    @once_differentiable
    def backward(ctx, do):
        _no_gradient(ctx, scale=5)
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
        # the same linear map, seen by autograd: it may be differentiated again
        return (Dropout.apply(dy, None, *ctx.how, ctx.per_row), dy if ctx.residual else None,
                None, None, None, None)
