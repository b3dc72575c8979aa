"""What the token operators refuse, in their C entries and in their binding, beyond the
shapes and pointers of test_tokens_abi.py (no GPU needed)."""
import ctypes as C
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
BAD = -1


def _attn(tok, **kw):
    s = dict(batch=2, q_heads=4, kv_heads=2, q_tokens=64, kv_tokens=64, dim=64, dtype=tok.BF16,
             causal=0, scale=0.125, spans_stride=0)
    s.update(kw)
    return tok._ATTN.pack(*s.values())


@pytest.mark.parametrize("dtype", ["BF16", "F16"])
@pytest.mark.parametrize("nq,nk", [(0, 64), (64, 64), (64, 0), (1, 8192)])
def test_backward_workspace_is_checked_whenever_there_is_one(tok, dtype, nq, nk):
    """Without queries too: whatever size is asked for is a pointer that will be written."""
    L, t = tok._lib(), tok._TOKENS.pack(1 << 20, 1 << 23, 512, 64)
    s = _attn(tok, dtype=getattr(tok, dtype), q_tokens=nq, kv_tokens=nk)
    need = L.gs_attention_bwd_workspace_size(s)
    if not need:
        return
    for ws in (None, C.c_void_p((1 << 20) + 16)):
        assert L.gs_attention_bwd(s, t, t, t, t, None, t, P, t, t, t, ws, need, None) == BAD
