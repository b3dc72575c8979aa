"""The token operators where results must not depend on what they do not see, at the ends of
their ranges, and on the paths that only large calls take, against the formulas in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

import token_reference as ref

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def _tokens():
    from gaussian_splatting_differentiable_amd import tokens
    return tokens


def _randn(seed, *shape, dtype=BF, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def _inputs(seed, B, nq, nk, H, Hk, d, dtype):
    return (_randn(seed, B, nq, H, d, dtype=dtype, scale=1.5), _randn(seed + 1, B, nk, Hk, d, dtype=dtype),
            _randn(seed + 2, B, nk, Hk, d, dtype=dtype), _randn(seed + 3, B, nq, H, d, dtype=dtype))


def _run(q, k, v, do, **how):
    tok = _tokens()
    o, lse = tok.attention(q, k, v, **how)
    dq, dk, dv = tok.attention_bwd(do, q, k, v, o, lse, **how)
    torch.cuda.synchronize()
    return dict(o=o, lse=lse, dq=dq, dk=dk, dv=dv)


def _compare(q, k, v, do, spans=None, causal=False, scale=None):
    allowed = ref.spans_of(q.shape[1], k.shape[1], spans, causal)
    want = ref.attention(q, k, v, allowed, scale or 1 / math.sqrt(q.shape[3]), do)
    got = _run(q, k, v, do, spans=spans, causal=causal, scale=scale)
    for n, x in got.items():
        ref.check(n, x, want[n])


def _list(*parts):
    """Spans of packed parts: (rows, lo, hi) each."""
    return torch.cat([torch.tensor([[lo, hi]], dtype=torch.int32).expand(n, 2)
                      for n, lo, hi in parts]).contiguous().cuda()


# ------------------------------------------------- fp16 gradients and what is not seen

def _lifted(seed, n, nk, H, Hk, d, lift):
    """Inputs whose q is `lift` times larger and k smaller: the scores are the same, and dk (or
    with 1 / lift dq) stays above fp16's smallest numbers where do is small."""
    q, k, v, do = _inputs(seed, 1, n, nk, H, Hk, d, FP)
    return q * lift, k / lift, v, do


@pytest.mark.parametrize("bad", [6e4, math.inf, math.nan])
@pytest.mark.parametrize("end", [1536, 1500])
@pytest.mark.parametrize("d,lift", [(64, 64.0), (64, 1 / 64), (128, 64.0), (128, 1 / 64)])
def test_small_gradients_beside_masked_places_in_fp16(bad, end, d, lift):
    """Padding in tiles of its own (1536) or inside one (1500), with gradients of 2^-17 beside."""
    q, k, v, do = _lifted(1, 1600, 1600, 2, 1, d, lift)
    do *= 2.0 ** -17
    for t in (q, k, v, do):
        t[:, end:] = bad
    _compare(q, k, v, do, spans=_list((end, 0, end), (1600 - end, 0, 0)))


@pytest.mark.parametrize("where", [64, 16383])
@pytest.mark.parametrize("bad", [6e4, math.inf])
def test_small_gradients_of_a_long_cache_with_a_masked_value_in_fp16(where, bad):
    """The value is in a tile that the queries see the rest of, or in one that none sees."""
    q, k, v, do = _lifted(2, 33, 16384, 1, 1, 64, 1 / 64)
    v[:, where] = bad
    spans = _list((33, 65, 16384)) if where == 64 else _list((33, 0, 16320))
    _compare(q, k, v, do * 2.0 ** -14, spans=spans)


@pytest.mark.parametrize("d", [64, 80, 128])
@pytest.mark.parametrize("lift", [64.0, 1 / 64])
def test_sequences_of_different_gradient_scales_in_fp16(d, lift):
    """Two packed sequences whose gradients are 2^22 apart, then their values 2^11."""
    q, k, v, do = _lifted(3, 1500, 1500, 2, 2, d, lift)
    do[:, :700] *= 2.0 ** -17
    do[:, 700:] *= 2.0 ** 5
    spans = _list((700, 0, 700), (800, 700, 1500))
    _compare(q, k, v, do, spans=spans)
    v[:, 700:] *= 2.0 ** 11
    do[:, 700:] *= 2.0 ** -16
    _compare(q, k, v, do, spans=spans)


def test_gradients_that_grow_and_shrink_along_the_tokens_in_fp16():
    """|do| over 2^16 from query to query and |v| over 2^8 from key to key, both ways (no result
    leaves fp16's range)."""
    for sign in (1, -1):
        q, k, v, do = _inputs(4, 1, 900, 900, 2, 1, 64, FP)
        ramp = 2.0 ** (sign * torch.linspace(-8, 8, 900, device="cuda"))[None, :, None, None]
        v = (v.float() * ramp.sqrt()).to(FP)
        do = (do.float() * ramp).to(FP)
        for causal in (False, True):
            allowed = ref.spans_of(900, 900, None, causal)
            want = ref.attention(q, k, v, allowed, 0.125, do)
            assert all(float(want[n][0].abs().max()) < 65504 for n in ("o", "dq", "dk", "dv"))
            _compare(q, k, v, do, causal=causal)


@pytest.mark.parametrize("nq,H", [(3, 1), (300, 64)])
def test_small_probabilities_of_a_long_row_in_fp16(nq, H):
    """One key holds nearly all of a row's probability, and 2^17 others 2^-26 of it each, which
    together are 2^-9: more than the result's rounding. Off by at most 2^-30 of the largest for
    each key (half the smallest number of fp16, and the 32-fold that p is held at)."""
    n = 1 << 17
    q = torch.zeros(1, nq, H, 64, dtype=FP, device="cuda")
    k = torch.zeros(1, n, 1, 64, dtype=FP, device="cuda")
    v = torch.ones(1, n, 1, 64, dtype=FP, device="cuda")
    q[..., 0], k[:, 77, :, 0], v[:, 77] = 4.0, 4.5, 0.0
    o, lse = _tokens().attention(q, k, v, scale=1.0)
    small = (n - 1) * math.exp(-18.0)
    want, room = small / (1 + small), n * 2.0 ** -30 + 4 * 2.0 ** -11 * small
    assert float((o.double() - want).abs().max()) <= room
    assert float((lse.double() - (18.0 + math.log1p(small))).abs().max()) <= 1e-5 * 18


# ------------------------------------------------- a NaN that is seen

def _time(call):
    call()
    best = math.inf
    for _ in range(3):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        a.record()
        call()
        b.record()
        b.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("mask", ["none", "causal", "packed"])
@pytest.mark.parametrize("where", ["value", "values", "all"])
def test_a_nan_that_is_seen_does_not_slow_a_call_down(mask, where):
    """A diverged step's NaN is there at the cost of a call, ten times at most, not that of every
    pair by itself: nothing masked has spoilt those rows, or they are NaN from the first key on."""
    tok = _tokens()
    q, k, v, do = _inputs(5, 1, 2048, 2048, 8, 8, 64, BF)
    how = dict(causal=mask == "causal",
               spans=_list((1000, 0, 1000), (1048, 1000, 2048)) if mask == "packed" else None)

    def step():
        o, lse = tok.attention(q, k, v, **how)
        return o, tok.attention_bwd(do, q, k, v, o, lse, **how)

    base = _time(step)
    if where == "value":
        v[:, 5] = math.nan
    elif where == "values":
        v.fill_(math.nan)
    else:
        for t in (q, k, v, do):
            t.fill_(math.nan)
    took = _time(step)
    o, (dq, dk, dv) = step()
    rows = torch.ones(2048, dtype=torch.bool, device="cuda")
    if where == "value":
        rows[:5] = mask != "causal"
        rows[1000:] = mask != "packed"
    for t in (o, dq):
        assert torch.equal(torch.isnan(t).all(3).all(2)[0], rows), mask
        assert torch.equal(torch.isnan(t).any(3).any(2)[0], rows), mask
    assert took <= 10 * base, (took, base)


@pytest.mark.parametrize("mask", ["none", "packed"])
@pytest.mark.parametrize("H,n", [(2, 300), (64, 300)])
def test_an_infinity_that_is_seen_with_the_smallest_probabilities(mask, H, n):
    """p v with p of about 2^-50, which is 0 in fp16, and an infinite v is infinite, not NaN; and
    so is p do in dv."""
    tok = _tokens()
    q, k, v, do = _inputs(15, 1, n, n, H, H, 64, FP)
    q[..., 0], k[..., 0] = 4.0, 0.0
    k[:, 20, :, 0] = -70.0  # a score of -35 beside those of the others
    v[:, 20, :, 7] = math.inf
    how = dict(spans=_list((n - 130, 0, n - 130), (130, n - 130, n)) if mask == "packed" else None)
    sees = n - 130 if mask == "packed" else n
    o, lse = tok.attention(q, k, v, **how)
    assert torch.all(o[:, :sees, :, 7] == math.inf) and torch.isfinite(o[:, sees:]).all()
    assert int((~torch.isfinite(o)).sum()) == sees * H
    v[:, 20, :, 7] = 0.5
    do[:, 30, :, 9] = math.inf
    o, lse = tok.attention(q, k, v, **how)
    _, _, dv = tok.attention_bwd(do, q, k, v, o, lse, **how)
    assert torch.all(dv[:, :sees, :, 9] == math.inf) and torch.isfinite(dv[:, sees:]).all()
    assert int((~torch.isfinite(dv)).sum()) == sees * H


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("H,nq,nk", [(2, 3, 9000), (6, 700, 700), (64, 150, 150)])
def test_a_masked_nan_beside_a_nan_that_is_seen(H, nq, nk, dtype):
    """Rows whose own NaN is in one element, in tiles where a masked key holds a NaN too, in the
    form for few rows (whole and in parts) and in that for many."""
    tok = _tokens()
    q, k, v, do = _inputs(16, 1, nq, nk, H, H // 2, 64, dtype)
    cut = nk - 100
    spans = _list((nq - 1, 0, cut), (1, cut, nk))  # the last query sees the last keys alone
    v[:, cut - 3, :, 5], v[:, cut + 2, :, 6] = math.nan, math.nan
    do[:, nq - 1, :, 8] = math.nan
    o, lse = tok.attention(q, k, v, spans=spans)
    bad = torch.zeros(1, nq, H, 64, dtype=torch.bool, device="cuda")
    bad[:, :nq - 1, :, 5], bad[:, nq - 1, :, 6] = True, True
    assert torch.equal(torch.isnan(o), bad)
    allowed = ref.spans_of(nq, nk, spans)
    clean = v.clone()
    clean[:, cut - 3, :, 5], clean[:, cut + 2, :, 6] = 0.0, 0.0
    want = ref.attention(q, k, clean, allowed, 0.125)
    ref.check("o", torch.where(bad, torch.zeros_like(o), o),
              (torch.where(bad.cpu(), 0.0, want["o"][0]), want["o"][1]))
    ref.check("lse", lse, want["lse"])
    # the gradients' NaN: a row's D is NaN with its o, so dq is, and dk of all that it sees
    dq, dk, dv = tok.attention_bwd(do, q, k, v, o, lse, spans=spans)
    assert torch.isnan(dq).all() and torch.isnan(dk).all()
    sees = torch.zeros(1, nk, H // 2, 64, dtype=torch.bool, device="cuda")
    sees[:, cut:, :, 8] = True
    assert torch.equal(torch.isnan(dv), sees)


# ------------------------------------------------- the ends of the ranges

@pytest.mark.parametrize("scale,by_q,by_k", [(2.0 ** -100, 2.0 ** 49, 2.0 ** 48),
                                             (2.0 ** 100, 2.0 ** -53, 2.0 ** -50)])
def test_scales_at_the_ends(scale, by_q, by_k):
    q, k, v, do = _inputs(6, 1, 150, 170, 2, 1, 64, BF)
    _compare(q * by_q, k * by_k, v, do, scale=scale)


@pytest.mark.parametrize("d,dtype", [(64, BF), (128, FP)])
def test_spans_with_so_many_blocks_that_one_pass_takes_both_sequences(d, dtype):
    """4096 blocks of rows: a block walks over the keys of both sequences that it has rows of."""
    B, H, n = 16, 128, 140
    q, k, v, do = _inputs(7, B, n, n, H, H, d, dtype)
    spans = _list((60, 0, 60), (50, 60, 110), (20, 105, 140), (10, 0, 0))
    got = _run(q, k, v, do, spans=spans)
    allowed = ref.spans_of(n, n, spans)
    for b, h in ((0, 0), (0, 127), (7, 61), (15, 3), (15, 127)):
        cut = [t[b:b + 1, :, h:h + 1] for t in (q, k, v, do)]
        want = ref.attention(*cut[:3], allowed, 1 / math.sqrt(d), cut[3])
        for name, x in got.items():
            ref.check(name, x[b:b + 1, h:h + 1] if name == "lse" else x[b:b + 1, :, h:h + 1],
                      want[name])


@pytest.mark.parametrize("mask", ["none", "late", "ends"])
@pytest.mark.parametrize("d,dtype", [(64, BF), (64, FP), (128, BF)])
def test_more_queries_than_a_block_of_keys_lists_at_a_time(mask, d, dtype):
    """2^18 + 70 queries of 40 keys: the keys' blocks walk twice over the tiles of queries. With
    all of them, with those of the second walk alone, and with a few of each."""
    n, nk = (1 << 18) + 70, 40
    q, k, v, do = _inputs(8, 1, n, nk, 1, 1, d, dtype)
    spans = {"none": None, "late": _list((1 << 18, 0, 0), (70, 0, nk)),
             "ends": _list((100, 3, nk), ((1 << 18) - 50, 0, 0), (20, 0, 17))}[mask]
    _compare(q, k, v, do, spans=spans)


# ------------------------------------------------- streams and autograd

def test_norm_and_rotation_on_another_stream_into_given_outputs():
    tok = _tokens()
    q, k = _randn(9, 2, 100, 4, 64), _randn(10, 2, 100, 2, 64)
    w = torch.rand(64).cuda() + 0.5
    want = tok.qk_norm_rope(q, k, w, w)
    grads = tok.qk_norm_rope_bwd(*want, q, k, w, w)
    s, outs = torch.cuda.Stream(), (torch.empty_like(q), torch.empty_like(k))
    s.wait_stream(torch.cuda.current_stream())
    got = tok.qk_norm_rope(q, k, w, w, q_out=outs[0], k_out=outs[1], stream=s)
    back = tok.qk_norm_rope_bwd(*got, q, k, w, w, stream=s)
    s.synchronize()
    assert got[0] is outs[0] and got[1] is outs[1]
    for a, b in zip((*got, *back), (*want, *grads)):
        assert torch.equal(a, b)


def test_autograd_of_queries_alone_and_of_dropped_rows():
    tok = _tokens()
    q, w = _randn(11, 1, 9, 4, 64), torch.rand(64).cuda() + 0.5
    xs = [t.clone().requires_grad_() for t in (q, w)]
    y, none = tok.QkNormRope.apply(xs[0], None, xs[1], None, None, None, False, 1e-6)
    assert none is None
    y.backward(torch.ones_like(y))
    dq, _, dw, _ = tok.qk_norm_rope_bwd(torch.ones_like(q), None, q, None, w, None)
    assert torch.equal(xs[0].grad, dq) and torch.equal(xs[1].grad, dw)
    x, r, g = (_randn(i, 20, 30) for i in (12, 13, 14))
    xs = [t.clone().requires_grad_() for t in (x, r)]
    tok.Dropout.apply(*xs, 0.4, 6, 7, True).backward(g)
    assert torch.equal(xs[0].grad, tok.dropout(g, 0.4, 6, 7, per_row=True))
    assert torch.equal(xs[1].grad, g)
