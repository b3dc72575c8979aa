"""The token operators' C entry points refuse bad arguments before any HIP call, and
their workspace sizes follow from the sizes (no GPU needed)."""
import ctypes as C
import math
import os

import pytest


@pytest.fixture(scope="module")
def tok():
    import gaussian_splatting_differentiable_amd as g
    if not os.path.exists(g.LIB_PATH):
        pytest.skip("libgs.so not built (run __graft_entry__.build())")
    from gaussian_splatting_differentiable_amd import tokens
    tokens._lib()
    return tokens


P = C.c_void_p(1 << 20)
BAD, WORKSPACE, UNSUPPORTED = -1, -3, -5


def _t(tok, at=1 << 20, b=1 << 16, t=512, h=64):
    return tok._TOKENS.pack(at, b, t, h)


def _attn(tok, **kw):
    s = dict(batch=2, q_heads=4, kv_heads=2, q_tokens=64, kv_tokens=64, dim=64, dtype=tok.BF16,
             causal=0, scale=0.125, spans_stride=0)
    s.update(kw)
    return tok._ATTN.pack(*s.values())


def _qk(tok, **kw):
    s = dict(batch=2, tokens=16, q_heads=4, k_heads=2, dim=64, dtype=tok.BF16, rot_dim=32,
             neighbours=0, n_positions=16, eps=1e-6, positions_stride=0)
    s.update(kw)
    return tok._QK.pack(*s.values())


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), BAD), (dict(q_tokens=-1), BAD), (dict(kv_heads=0), BAD),
    (dict(q_heads=3), BAD), (dict(dim=0), BAD), (dict(dim=60), UNSUPPORTED),
    (dict(dim=136), UNSUPPORTED), (dict(dtype=0), UNSUPPORTED), (dict(dtype=7), BAD),
    (dict(causal=2), BAD), (dict(scale=0.0), BAD), (dict(scale=math.inf), BAD),
    (dict(scale=math.nan), BAD), (dict(spans_stride=-1), BAD),
    (dict(kv_tokens=1 << 30), UNSUPPORTED), (dict(batch=1 << 29), UNSUPPORTED)])
def test_attention_shapes(tok, kw, status):
    L, t, s = tok._lib(), _t(tok), _attn(tok, **kw)
    big = 1 << 40
    assert L.gs_attention(s, t, t, t, None, t, P, P, big, None) == status
    assert L.gs_attention_bwd(s, t, t, t, t, None, t, P, t, t, t, P, big, None) == status
    assert L.gs_attention_workspace_size(s) == 0
    assert L.gs_attention_bwd_workspace_size(s) == 0


@pytest.mark.parametrize("kw", [
    dict(batch=1 << 18, q_heads=32, kv_heads=32, q_tokens=1, kv_tokens=1), dict(batch=1 << 21),
    dict(batch=1, q_heads=1, kv_heads=1, q_tokens=1, kv_tokens=(1 << 29) + 1)])
def test_attention_launches_too_large(tok, kw):
    """More rows than a launch has threads for are refused, not left to the launch."""
    L, t, s = tok._lib(), _t(tok, t=8), _attn(tok, **kw)
    assert L.gs_attention(s, t, t, t, None, t, P, P, 1 << 50, None) == UNSUPPORTED
    assert L.gs_attention_bwd(s, t, t, t, t, None, t, P, t, t, t, P, 1 << 50, None) == UNSUPPORTED
    assert L.gs_attention_workspace_size(s) == 0


def test_qk_launches_too_large(tok):
    L, t = tok._lib(), _t(tok)
    s = _qk(tok, batch=1 << 14, tokens=1 << 14, q_heads=8, rot_dim=0)
    assert L.gs_qk_norm_rope(s, t, t, None, None, None, None, t, t, None) == UNSUPPORTED


def test_attention_pointers_strides_and_workspace(tok):
    L, t, s = tok._lib(), _t(tok), _attn(tok)
    big = 1 << 40

    def fwd(q=t, k=t, v=t, spans=None, o=t, lse=P, ws=P, size=big, shape=s):
        return L.gs_attention(shape, q, k, v, spans, o, lse, ws, size, None)

    assert L.gs_attention(None, t, t, t, None, t, P, P, big, None) == BAD
    for name in "qkvo":
        assert fwd(**{name: None}) == BAD
        assert fwd(**{name: _t(tok, at=0)}) == BAD
        assert fwd(**{name: _t(tok, at=(1 << 20) + 8)}) == BAD
        assert fwd(**{name: _t(tok, t=516)}) == BAD
        assert fwd(**{name: _t(tok, h=-64)}) == BAD
        assert fwd(**{name: _t(tok, t=1 << 23)}) == UNSUPPORTED
    assert fwd(o=_t(tok, t=0)) == BAD                       # outputs may not overlap
    assert fwd(lse=None) == BAD
    assert fwd(spans=C.c_void_p((1 << 20) + 4)) == BAD
    few = _attn(tok, q_tokens=1, kv_tokens=8192)
    need = L.gs_attention_workspace_size(few)
    assert need > 0
    assert fwd(shape=few, size=need - 1) == WORKSPACE
    assert fwd(shape=few, ws=None) == BAD
    assert fwd(shape=few, ws=C.c_void_p((1 << 20) + 16)) == BAD
    need = L.gs_attention_bwd_workspace_size(s)
    assert need >= 2 * 4 * 64 * 4
    bwd = lambda **kw: L.gs_attention_bwd(
        s, t, t, t, t, None, kw.get("o", t), kw.get("lse", P), kw.get("dq", t), t, kw.get("dv", t),
        kw.get("ws", P), kw.get("size", big), None)
    assert bwd(size=need - 1) == WORKSPACE
    assert bwd(ws=None) == BAD and bwd(lse=None) == BAD and bwd(dq=None) == BAD
    assert bwd(dv=_t(tok, h=0)) == BAD and bwd(o=None) == BAD


def test_nothing_to_do_is_ok(tok):
    L = tok._lib()
    for kw in (dict(batch=0), dict(q_tokens=0)):
        s = _attn(tok, **kw)
        t = None if "batch" in kw else _t(tok)
        assert L.gs_attention(s, None, t, t, None, None, None, None, 0, None) == 0
    assert L.gs_qk_norm_rope(_qk(tok, tokens=0, rot_dim=0), None, None, None, None, None, None,
                             None, None, None) == 0
    assert L.gs_dropout(0, 5, 0, None, 0, None, 0, None, 0, 0.5, 1, 2, 0, None) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), BAD), (dict(dim=0), BAD), (dict(dim=60), UNSUPPORTED),
    (dict(dim=264), UNSUPPORTED), (dict(rot_dim=72), BAD), (dict(rot_dim=12), UNSUPPORTED),
    (dict(rot_dim=-8), BAD), (dict(dtype=3), BAD), (dict(neighbours=2), BAD), (dict(eps=-1.0), BAD),
    (dict(eps=math.nan), BAD), (dict(n_positions=-1), BAD), (dict(positions_stride=-1), BAD),
    (dict(q_heads=65536), UNSUPPORTED)])
def test_qk_shapes(tok, kw, status):
    L, t, s = tok._lib(), _t(tok), _qk(tok, **kw)
    assert L.gs_qk_norm_rope(s, t, t, None, None, P, None, t, t, None) == status
    assert L.gs_qk_norm_rope_bwd(s, t, t, t, t, None, None, P, None, t, t, None, None, None, 0,
                                 None) == status
    assert L.gs_qk_workspace_size(s) == 0


def test_qk_pointers_and_workspace(tok):
    L, t, s = tok._lib(), _t(tok), _qk(tok)
    odd = C.c_void_p((1 << 20) + 8)
    assert L.gs_qk_norm_rope(s, None, t, None, None, P, None, t, t, None) == BAD
    assert L.gs_qk_norm_rope(s, t, t, odd, None, P, None, t, t, None) == BAD
    assert L.gs_qk_norm_rope(s, t, t, None, None, odd, None, t, t, None) == BAD
    assert L.gs_qk_norm_rope(s, t, t, None, None, None, None, t, t, None) == BAD
    assert L.gs_qk_norm_rope(s, t, t, None, None, P, C.c_void_p(6), t, t, None) == BAD
    assert L.gs_qk_norm_rope(_qk(tok, n_positions=15), t, t, None, None, P, None, t, t, None) == BAD
    need = L.gs_qk_workspace_size(s)
    assert need > 0
    back = lambda ws, size: L.gs_qk_norm_rope_bwd(s, t, t, t, t, None, None, P, None, t, t, P, None,
                                                  ws, size, None)
    assert back(P, need - 1) == WORKSPACE and back(None, need) == BAD


def test_dropout_arguments(tok):
    L = tok._lib()
    call = lambda rows=4, cols=8, dt=0, x=P, xs=8, r=None, rs=0, y=P, ys=8, p=0.5, row=0: \
        L.gs_dropout(rows, cols, dt, x, xs, r, rs, y, ys, p, 1, 2, row, None)
    assert call(rows=-1) == BAD and call(dt=5) == BAD and call(p=1.0) == BAD
    assert call(p=math.nan) == BAD and call(row=2) == BAD and call(x=None) == BAD
    assert call(y=C.c_void_p((1 << 20) + 2)) == BAD and call(ys=7) == BAD and call(xs=-8) == BAD
    assert call(rows=1 << 41) == UNSUPPORTED
