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


def _qk_norm_rope(q, k, q_weight=None, k_weight=None, *, cos_sin=None, positions=None,
                  neighbours=False, eps=1e-6):
    return _norm(q, q_weight, eps), _norm(k, k_weight, eps)


def _qk_norm_rope_bwd(dq_out, dk_out, q, k, q_weight=None, k_weight=None, *, cos_sin=None,
                      positions=None, neighbours=False, eps=1e-6):
    dq, dqw = (None, None) if q is None else _norm_bwd(dq_out, q, q_weight, eps)
    dk, dkw = (None, None) if k is None else _norm_bwd(dk_out, k, k_weight, eps)
    return dq, dk, dqw, dkw


def _attention(q, k, v, *, spans=None, causal=False, scale=None):
    s = torch.einsum("bnhd,bmhd->bhnm", q, k) * (1.0 if scale is None else scale)
    return torch.einsum("bhnm,bmhd->bnhd", torch.softmax(s, 3), v), torch.logsumexp(s, 3)


def _attention_bwd(do, q, k, v, o, lse, **how):
    with torch.enable_grad():
        xs = [t.detach().requires_grad_() for t in (q, k, v)]
        y, _ = _attention(*xs, **how)
    return torch.autograd.grad(y, xs, do)


def _dropout(x, p, seed, offset=0, *, residual=None, per_row=False):
    g = torch.Generator().manual_seed(seed + offset)
    keep = torch.rand(x.shape[:1] if per_row else x.shape, generator=g) >= p
    keep = keep.view(-1, *[1] * (x.dim() - 1)) if per_row else keep
    y = torch.where(keep, x / (1 - p), torch.zeros(()))
    return y if residual is None else residual + y


@pytest.fixture
def tok(monkeypatch):
    """The module, its calls stood in for by the formulas, whose inside autograd does not see."""
    from gaussian_splatting_differentiable_amd import tokens

    def opaque(f):
        def call(*args, **kw):
            with torch.no_grad():
                return f(*args, **kw)
        return call

    for f in (_qk_norm_rope, _qk_norm_rope_bwd, _attention, _attention_bwd, _dropout):
        monkeypatch.setattr(tokens, f.__name__[1:], opaque(f))
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


def _square_of_gradient(f, x, w):
    """|d/dx |f(x w)|^2|^2: w is in it both through f and beside it."""
    g, = torch.autograd.grad(f(x * w).square().sum(), x, create_graph=True)
    return g.square().sum()


def test_second_derivatives_are_refused_not_dropped(tok):
    """Attention and the norm have no second derivative: asking for one is an error, where a
    backward that autograd does not see would leave its terms out of the result."""
    x, w = _randn(4, 1, 3, 2, 8).requires_grad_(), _randn(5, 8).requires_grad_()
    k, v = _randn(6, 1, 4, 2, 8), _randn(7, 1, 4, 2, 8)
    for f in (lambda q: tok.Attention.apply(q, k, v, None, False, None),
              lambda q: tok.QkNormRope.apply(q, k, None, None, None, None, False, 1e-6)[0]):
        with pytest.raises(RuntimeError, match="differentiate twice"):
            _square_of_gradient(f, x, w).backward()


@pytest.mark.parametrize("per_row", [False, True])
@pytest.mark.parametrize("residual", [False, True])
def test_dropout_is_differentiable_twice(tok, per_row, residual):
    x, w, r = (_randn(i, 5, 7).requires_grad_() for i in (8, 9, 10))
    rest = (r,) if residual else ()

    def second(f):
        return torch.autograd.grad(_square_of_gradient(f, x, w), (x, w, *rest))

    got = second(lambda t: tok.Dropout.apply(t, *(rest or (None,)), 0.4, 3, 5, per_row))
    want = second(lambda t: _dropout(t, 0.4, 3, 5, residual=r if rest else None, per_row=per_row))
    for a, b in zip(got, want):
        assert torch.allclose(a, b, rtol=1e-12, atol=1e-12)


def test_a_scale_that_changes_between_forward_and_backward(tok):
    """The backward belongs to the forward that was made."""
    q, k, v = (_randn(i, 1, 3, 2, 8).requires_grad_() for i in (11, 12, 13))
    scale, eps = torch.tensor(0.5, dtype=torch.float64), torch.tensor(0.25, dtype=torch.float64)
    y = tok.Attention.apply(q, k, v, None, False, scale)
    a, _ = tok.QkNormRope.apply(q, None, None, None, None, None, False, eps)
    scale += 1.0
    eps += 1.0
    got = torch.autograd.grad(y.sum() + a.square().sum(), q)[0]
    y, _ = _attention(q, k, v, scale=0.5)
    want = torch.autograd.grad(y.sum() + _norm(q, None, 0.25).square().sum(), q)[0]
    assert torch.allclose(got, want, rtol=1e-12, atol=1e-12)


def test_what_gets_no_gradient_may_not_want_one(tok):
    """A learned table, eps or scale would stay as it is without a word."""
    x, table = _randn(14, 1, 3, 2, 8).requires_grad_(), _randn(15, 3, 8)
    number = torch.tensor(0.5, dtype=torch.float64)

    def norm(table, eps):
        return tok.QkNormRope.apply(x, None, None, None, table, None, False, eps)

    def attention(scale):
        return tok.Attention.apply(x, x, x, None, False, scale)

    wants = table.clone().requires_grad_(), number.clone().requires_grad_()
    for call, arg, want in ((lambda t: norm(t, 1e-6), table, wants[0]),
                            (lambda t: norm(None, t), number, wants[1]),
                            (attention, number, wants[1])):
        y = call(arg)
        (y[0] if isinstance(y, tuple) else y).sum().backward()
        y = call(want)
        with pytest.raises(ValueError, match="no gradient"):
            (y[0] if isinstance(y, tuple) else y).sum().backward()
        with torch.no_grad():
            call(want)


def test_an_output_that_overwrites_what_autograd_saved_is_noticed(tok):
    """An output that the caller gives is written like any in-place result."""
    base = _randn(16, 3, 4)
    w = _randn(17, 4).requires_grad_()
    for part in (base, base[1:]):
        y = (base * w).sum()
        assert tok._out("out", part, part) is part  # as every call takes its outputs
        with pytest.raises(RuntimeError, match="modified by an inplace operation"):
            y.backward()
    with torch.inference_mode():
        x = torch.zeros(3)
        assert tok._out("out", x, x) is x
