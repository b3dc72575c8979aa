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
BAD, UNSUPPORTED = -1, -5


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


def test_every_tensor_of_a_call_is_marked_as_used_on_its_stream(tok, monkeypatch):
    """What the caller gives for outputs too: memory that it drops while the other stream still
    writes there must not be handed out again."""
    torch = pytest.importorskip("torch")

    class Left(Exception):
        pass

    def there(stream, device, tensors):
        marked.extend(id(t) for t in tensors if t is not None)
        raise Left

    monkeypatch.setattr(tok, "_elsewhere", lambda stream, device: True)
    monkeypatch.setattr(tok, "_there", there)
    monkeypatch.setattr(tok, "_qk_args", lambda *a: (None, 0, None, None, [None] * 4, None))
    monkeypatch.setattr(tok, "_attn_args", lambda *a: (None, (None, (1, 2, 3), 0, 0)))
    monkeypatch.setattr(tok, "_DTYPES", {torch.float32: 0})

    def t(*shape):
        return torch.zeros(*shape)

    class OnDevice:  # dropout looks at its input's device before anything else
        device, dtype = torch.device("cuda", 0), torch.float32

    x = (1, 3, 2, 8)
    calls = [
        (tok.qk_norm_rope, [t(*x), t(*x), t(8), t(8)],
         dict(cos_sin=t(3, 8), positions=t(3), q_out=t(*x), k_out=t(*x))),
        (tok.qk_norm_rope_bwd, [t(*x), t(*x), t(*x), t(*x), t(8), t(8)],
         dict(cos_sin=t(3, 8), positions=t(3))),
        (tok.attention, [t(*x), t(*x), t(*x)], dict(spans=t(3, 2), out=t(*x), workspace=t(64))),
        (tok.attention_bwd, [t(*x), t(*x), t(*x), t(*x), t(*x), t(1, 2, 3)],
         dict(spans=t(3, 2), workspace=t(64))),
        (tok.dropout, [OnDevice()], dict(p=0.5, seed=1, residual=t(*x), out=t(*x))),
    ]
    for call, args, kw in calls:
        marked = []
        with pytest.raises(Left):
            call(*args, **kw, stream=object())
        for a in args + [v for v in kw.values() if isinstance(v, torch.Tensor)]:
            assert id(a) in marked, (call.__name__, getattr(a, "shape", a))


def test_a_stream_of_another_device_is_refused(tok):
    """Its work would otherwise run on the current stream of the tensors' device, unordered with
    what the caller has on the one that it named."""
    torch = pytest.importorskip("torch")

    class Stream:
        device = torch.device("cuda", 1)

    assert tok._elsewhere(Stream(), torch.device("cuda", 1))
    with pytest.raises(ValueError):
        tok._elsewhere(Stream(), torch.device("cuda", 0))


def test_a_scale_or_eps_that_changes_in_place_is_read_at_every_call(tok):
    """What a call keeps for its sizes is kept by their values, not by the object that held one."""
    torch = pytest.importorskip("torch")

    class Tensor:
        device, dtype = torch.device("cuda", 0), torch.bfloat16

        def __init__(self, *shape):
            self.shape = torch.Size(shape)

        def dim(self):
            return len(self.shape)

        def stride(self):
            return (1 << 12, 1 << 8, self.shape[-1], 1)

        def data_ptr(self):
            return 1 << 20

    x = Tensor(1, 3, 2, 64)
    for number in (torch.tensor(0.5), __import__("numpy").array(0.5)):
        a = tok._attn_args(x, x, x, None, False, number)[1][0]
        e = tok._qk_args(x, x, None, None, None, None, False, number)[0]
        number += 0.25
        b = tok._attn_args(x, x, x, None, False, number)[1][0]
        f = tok._qk_args(x, x, None, None, None, None, False, number)[0]
        assert tok._ATTN.unpack(a)[8] == tok._QK.unpack(e)[9] == 0.5
        assert tok._ATTN.unpack(b)[8] == tok._QK.unpack(f)[9] == 0.75


def test_scales_whose_log_sums_leave_32_bits_are_refused(tok):
    """The backward starts its scores from -lse / scale, the forward multiplies by scale log2 e:
    both stay finite for scales from 2^-100 to 2^100."""
    L, t = tok._lib(), tok._TOKENS.pack(1 << 20, 1 << 23, 512, 64)
    for scale in (2.0 ** -101, 1e-38, 1e-45, 2.0 ** 101, 3e38):
        s = _attn(tok, scale=scale)
        assert L.gs_attention(s, t, t, t, None, t, P, P, 1 << 40, None) == UNSUPPORTED
        assert L.gs_attention_bwd(s, t, t, t, t, None, t, P, t, t, t, P, 1 << 40, None) == UNSUPPORTED
        assert L.gs_attention_bwd_workspace_size(s) == 0
    for scale in (2.0 ** -100, 2.0 ** 100):
        assert L.gs_attention_bwd_workspace_size(_attn(tok, scale=scale)) > 0
