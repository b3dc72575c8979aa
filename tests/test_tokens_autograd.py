"""The token operators' autograd classes on the CPU: the calls they make are stood in for
by torch formulas, so that what is tested is what the classes do with them."""
import pytest

torch = pytest.importorskip("torch")


def _norm(x, w, eps):
    if x is None:
        return None
    y = x / (x.square().mean(3, keepdim=True) + eps).sqrt()
    return y if w is None else y * w


def _norm_bwd(dy, x, w, eps):
    with torch.enable_grad():
        xs = [t.detach().requires_grad_() for t in (x, w) if t is not None]
        y = _norm(xs[0], xs[1] if w is not None else None, eps)
    g = torch.autograd.grad(y, xs, dy)
    return g[0], g[1] if w is not None else None


@pytest.fixture
def tok(monkeypatch):
    from gaussian_splatting_differentiable_amd import tokens

    def qk_norm_rope(q, k, q_weight=None, k_weight=None, *, cos_sin=None, positions=None,
                     neighbours=False, eps=1e-6):
        return _norm(q, q_weight, eps), _norm(k, k_weight, eps)

    def qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, *, cos_sin=None,
                         positions=None, neighbours=False, eps=1e-6):
        dq, dqw = (None, None) if q is None else _norm_bwd(dq_out, q, q_weight, eps)
        dk, dkw = (None, None) if k is None else _norm_bwd(dk_out, k, k_weight, eps)
        return dq, dk, dqw, dkw

    def attention(q, k, v, *, spans=None, causal=False, scale=None):
        s = torch.einsum("bnhd,bmhd->bhnm", q, k) * (1.0 if scale is None else scale)
        p = torch.softmax(s, 3)
        return torch.einsum("bhnm,bmhd->bnhd", p, v), torch.logsumexp(s, 3)

    def attention_bwd(do, q, k, v, o, lse, **how):
        with torch.enable_grad():
            xs = [t.detach().requires_grad_() for t in (q, k, v)]
            y, _ = attention(*xs, **how)
        return torch.autograd.grad(y, xs, do)

    def dropout(x, p, seed, offset=0, *, residual=None, per_row=False):
        g = torch.Generator().manual_seed(seed + offset)
        keep = torch.rand(x.shape[:1] if per_row else x.shape, generator=g) >= p
        keep = keep.view(-1, *[1] * (x.dim() - 1)) if per_row else keep
        y = torch.where(keep, x / (1 - p), torch.zeros(()))
        return y if residual is None else residual + y

    for f in (qk_norm_rope, qk_norm_rope_bwd, attention, attention_bwd, dropout):
        monkeypatch.setattr(tokens, f.__name__, f)
    return tokens


def _randn(seed, *shape):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed), dtype=torch.float64)


@pytest.mark.parametrize("which", ["queries", "keys"])
def test_queries_or_keys_alone(tok, which):
    x, w, g = _randn(1, 2, 3, 4, 8).requires_grad_(), _randn(2, 8).requires_grad_(), _randn(3, 2, 3, 4, 8)
    if which == "queries":
        y, other = tok.QkNormRope.apply(x, None, w, None, None, None, False, 1e-6)
    else:
        other, y = tok.QkNormRope.apply(None, x, None, w, None, None, False, 1e-6)
    assert other is None
    y.backward(g)
    want = _norm_bwd(g, x, w, 1e-6)
    assert torch.equal(x.grad, want[0]) and torch.equal(w.grad, want[1])
