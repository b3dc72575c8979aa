"""Dropout from the counter-based generator (gs_dropout): the mask word for word
against the generator in Python integers, the values against the formula."""
import math

import pytest

torch = pytest.importorskip("torch")

import token_reference as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _tokens():
    from gaussian_splatting_differentiable_amd import tokens
    return tokens


def _randn(seed, *shape, dtype=torch.float32):
    return torch.randn(shape, generator=torch.Generator().manual_seed(seed)).to(dtype).cuda()


def _want(x, p, seed, offset, residual, per_row):
    rows, cols = (x.numel() // x.shape[-1], x.shape[-1]) if x.dim() > 1 else (1, x.numel())
    words = torch.tensor(ref.philox(rows if per_row else rows * cols, seed, offset),
                         dtype=torch.int64)
    keep = words >= round(p * 2 ** 32)
    keep = keep.repeat_interleave(cols) if per_row else keep
    keep = keep.view(x.shape)
    y = torch.where(keep, x.cpu().double() / (1 - p), torch.zeros((), dtype=torch.float64))
    r = torch.zeros_like(y) if residual is None else residual.cpu().double()
    u = ref.U[x.dtype]
    # the scale, the product and the sum in 32 bits, then one rounding to the type
    room = 4 * 2.0 ** -24 * (y.abs() + r.abs()) + 1.01 * u * (y + r).abs() + ref.TINY[x.dtype]
    return y + r, room, keep


def _compare(x, p=0.3, seed=1234567890123, offset=0, residual=None, per_row=False):
    y = _tokens().dropout(x, p, seed, offset, residual=residual, per_row=per_row)
    value, room, keep = _want(x, p, seed, offset, residual, per_row)
    ref.check("y", y, (value, room))
    if residual is None:
        assert not y.cpu()[~keep].any()
    return y


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 7), (5, 1), (16, 64), (33, 3), (7, 333),
                                       (3, 1000), (600, 8), (1030, 1)])
@pytest.mark.parametrize("res", [False, True])
@pytest.mark.parametrize("per_row", [False, True])
def test_sizes(dtype, rows, cols, res, per_row):
    x = _randn(1, rows, cols, dtype=dtype)
    _compare(x, residual=_randn(2, rows, cols, dtype=dtype) if res else None, per_row=per_row)


@pytest.mark.parametrize("seed,offset", [(0, 0), (2 ** 64 - 1, 5), (7, 2 ** 32 - 3),
                                         (1 << 40, 2 ** 64 - 20), (-1, 3)])
def test_seeds_and_counters_past_32_and_at_64_bits(seed, offset):
    x = _randn(3, 5, 40)
    y = _tokens().dropout(x, 0.5, seed, offset)
    value, room, _ = _want(x, 0.5, seed % 2 ** 64, offset, None, False)
    ref.check("y", y, (value, room))


def test_generator_against_published_words():
    """The first block of key 0, counter 0, as printed with the generator's publication
    (known-answer vector of Philox 4x32-10)."""
    assert ref.philox(4, 0, 0) == [0x6627e8d5, 0xe169c58d, 0xbc57ac4c, 0x9b00dbd8]


@pytest.mark.parametrize("p", [0.0, 1e-9, 0.1, 0.9999999, 1.0 - 2.0 ** -40])
def test_probabilities_at_the_ends(p):
    x = _randn(4, 64, 64)
    y = _tokens().dropout(x, p, 9)
    if p == 0.0:
        assert torch.equal(x, y)
    value, room, keep = _want(x, p, 9, 0, None, False)
    if p < 0.99:
        ref.check("y", y, (value, room))
    else:
        assert int((y != 0).sum()) <= 2


def test_kept_share_and_mean():
    """A million draws: the kept share within five standard deviations of 1 - p."""
    n, p = 1 << 20, 0.3
    y = _tokens().dropout(torch.ones(n // 64, 64, device="cuda"), p, 77, 1 << 35)
    kept = float((y != 0).double().mean())
    assert abs(kept - (1 - p)) < 5 * math.sqrt(p * (1 - p) / n)


def test_dropped_nan_and_infinity_are_gone():
    x = _randn(5, 32, 32)
    _, _, keep = _want(x, 0.5, 3, 0, None, False)
    x[~keep.cuda()] = math.nan
    x[0][~keep[0].cuda()] = math.inf
    y = _tokens().dropout(x, 0.5, 3)
    assert torch.isfinite(y).all() and not y[~keep.cuda()].any()


@pytest.mark.parametrize("per_row", [False, True])
def test_strides_alignment_and_in_place(per_row):
    """Column slices, rows off 16-byte boundaries and results in place draw the same mask."""
    tok = _tokens()
    x = _randn(6, 50, 64, dtype=torch.bfloat16)
    want = tok.dropout(x, 0.25, 8, 2, per_row=per_row)
    wide = torch.zeros(50, 100, dtype=torch.bfloat16, device="cuda")
    wide[:, 3:67] = x
    out = torch.full((50, 90), 5.0, dtype=torch.bfloat16, device="cuda")
    tok.dropout(wide[:, 3:67], 0.25, 8, 2, per_row=per_row, out=out[:, 11:75])
    assert torch.equal(out[:, 11:75], want)
    assert torch.all(out[:, :11] == 5) and torch.all(out[:, 75:] == 5)
    col = torch.zeros(50, 7, device="cuda")
    col[:, 2] = _randn(7, 50)
    a = tok.dropout(col[:, 2:3], 0.5, 1, per_row=per_row)
    assert torch.equal(a, tok.dropout(col[:, 2:3].contiguous(), 0.5, 1, per_row=per_row))
    tok.dropout(x, 0.25, 8, 2, per_row=per_row, out=x)
    assert torch.equal(x, want)


def test_parts_of_a_draw_and_more_than_2_32_elements():
    """Counters continue: a part from its own offset equals that part of the whole; and the
    element index passes 32 bits."""
    tok = _tokens()
    x = _randn(8, 8, 64)
    whole = tok.dropout(x, 0.5, 4, 10)
    assert torch.equal(tok.dropout(x[4:], 0.5, 4, 10 + 4 * 64 // 4), whole[4:])
    n = (1 << 32) + 64
    big = torch.ones(n // 64, 64, dtype=torch.float16, device="cuda")
    tok.dropout(big, 0.5, 4, 10, out=big)
    tail = tok.dropout(torch.ones(2, 64, dtype=torch.float16, device="cuda"), 0.5, 4,
                       10 + (n - 128) // 4)
    assert torch.equal(big[-2:], tail)


def test_gradient_is_the_same_map():
    """y is linear in x: <dropout(x), g> = <x, dropout(g)>, and autograd gives it."""
    tok = _tokens()
    x, r, g = _randn(9, 20, 30), _randn(10, 20, 30), _randn(11, 20, 30)
    xs = [t.clone().requires_grad_() for t in (x, r)]
    y = tok.Dropout.apply(*xs, 0.4, 6, 7, False)
    y.backward(g)
    dx = tok.dropout(g, 0.4, 6, 7)
    assert torch.equal(xs[0].grad, dx) and torch.equal(xs[1].grad, g)
    a = float((tok.dropout(x, 0.4, 6, 7).double() * g.double()).sum())
    b = float((x.double() * dx.double()).sum())
    room = 4 * 2.0 ** -24 * float((x.double() * dx.double()).abs().sum())
    assert abs(a - b) <= room
    h = 2.0 ** -3
    t = _randn(12, 20, 30)
    up = tok.dropout(x + h * t, 0.4, 6, 7, residual=r).double()
    down = tok.dropout(x - h * t, 0.4, 6, 7, residual=r).double()
    diff = float(((up - down) / (2 * h) * g.double()).sum())
    size = float((g.abs() * (x.abs() + t.abs() + r.abs())).sum()) * 2
    assert abs(diff - float((dx.double() * t.double()).sum())) <= 8 * 2.0 ** -24 * size / h


def test_refusals():
    import gaussian_splatting_differentiable_amd as gsr
    tok = _tokens()
    x = _randn(13, 4, 8)
    for p in (1.0, -0.1, math.nan, 2.0):
        with pytest.raises(gsr.GsError) as e:
            tok.dropout(x, p, 1)
        assert e.value.status == gsr.GS_ERR_INVALID_ARGUMENT
    for f in (lambda: tok.dropout(x, 0.1, 1, residual=x.half()), lambda: tok.dropout(x.cpu(), 0.1, 1),
              lambda: tok.dropout(x, 0.1, 1, residual=x[:2]), lambda: tok.dropout(x.t(), 0.1, 1),
              lambda: tok.dropout(x[0], 0.1, 1, per_row=True), lambda: tok.dropout(x.long(), 0.1, 1)):
        with pytest.raises(ValueError):
            f()
    assert tok.dropout(x[:0], 0.1, 1).numel() == 0
