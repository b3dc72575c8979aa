"""Attention and its gradient (gs_attention, gs_attention_bwd) against the formulas
in 64 bits, at the sizes, masks and layouts where kernels of this kind go wrong."""
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


def _compare(q, k, v, do, spans=None, causal=False, scale=None):
    tok = _tokens()
    nq, nk = q.shape[1], k.shape[1]
    allowed = ref.spans_of(nq, nk, spans, causal)
    want = ref.attention(q, k, v, allowed, scale or 1 / math.sqrt(q.shape[3]), do)
    how = dict(spans=spans, causal=causal, scale=scale)
    o, lse = tok.attention(q, k, v, **how)
    got = dict(o=o, lse=lse)
    if do is not None:
        got["dq"], got["dk"], got["dv"] = tok.attention_bwd(do, q, k, v, o, lse, **how)
    torch.cuda.synchronize()
    for n, x in got.items():
        ref.check(n, x, want[n])
    return got


# one token, ends inside and at the edges of tiles of 32, 64 and 128, odd sizes
SIZES = [(1, 1, 1), (1, 1, 200), (2, 1, 64), (1, 3, 33), (1, 31, 32), (2, 32, 65), (1, 63, 63),
         (1, 64, 128), (1, 65, 1), (1, 128, 127), (2, 129, 257), (1, 300, 300), (1, 200, 513)]


@pytest.mark.parametrize("B,nq,nk", SIZES)
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, BF), (80, FP)])
def test_sizes(B, nq, nk, d, dtype):
    _compare(*_inputs(1, B, nq, nk, 4, 2, d, dtype))


@pytest.mark.parametrize("nq,nk", [(1, 1), (5, 130), (130, 5), (200, 200), (129, 300)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_causal(nq, nk, dtype):
    """Queries aligned with the last keys; with more queries than keys the first see none."""
    _compare(*_inputs(2, 2, nq, nk, 4, 4, 64, dtype), causal=True)


@pytest.mark.parametrize("d", [8, 16, 24, 40, 56, 64, 72, 96, 104, 120, 128])
@pytest.mark.parametrize("nq", [7, 140])
def test_head_sizes(d, nq):
    _compare(*_inputs(3, 1, nq, 150, 2, 1, d, BF))


@pytest.mark.parametrize("H,Hk", [(1, 1), (3, 3), (6, 2), (8, 1), (7, 1), (40, 1), (5, 5)])
@pytest.mark.parametrize("nq", [1, 9, 140])
def test_shared_heads(H, Hk, nq):
    _compare(*_inputs(4, 2, nq, 170, H, Hk, 64, BF))


@pytest.mark.parametrize("B,H,nq,nk", [(1, 64, 129, 129), (4, 32, 150, 70), (16, 16, 40, 200)])
@pytest.mark.parametrize("d", [64, 128])
def test_many_workgroups(B, H, nq, nk, d):
    """Enough heads for the form that takes many rows, with rows past its tiles' ends."""
    _compare(*_inputs(5, B, nq, nk, H, H // 2, d, BF))


def _random_spans(seed, B, nq, nk):
    g = torch.Generator().manual_seed(seed)
    a = torch.randint(-3, nk + 1, (B, nq), generator=g)
    n = torch.randint(0, nk // 2 + 2, (B, nq), generator=g)
    n[:, ::7] = 0                        # rows that see nothing
    n[:, 3::11] = 1                      # and rows that see one key
    return torch.stack([a, a + n], 2).int().cuda()


@pytest.mark.parametrize("nq,nk", [(1, 40), (90, 200), (300, 260)])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("d,dtype", [(64, BF), (128, FP)])
def test_spans(nq, nk, causal, d, dtype):
    _compare(*_inputs(6, 2, nq, nk, 4, 2, d, dtype), spans=_random_spans(7, 2, nq, nk),
             causal=causal)


@pytest.mark.parametrize("H", [4, 64])
def test_packed_sequences_share_one_span_list(H):
    """Sequences of 1, 70, 64 and 100 tokens in one row, then padding; one list for the batch."""
    cuts, n = [0, 1, 71, 135, 235], 260
    spans = torch.zeros(n, 2, dtype=torch.int32)
    for a, b in zip(cuts, cuts[1:]):
        spans[a:b, 0], spans[a:b, 1] = a, b
    got = _compare(*_inputs(8, 2, n, n, H, H, 64, BF), spans=spans.cuda())
    assert not got["o"][:, 235:].any() and torch.all(got["lse"][:, :, 235:] == -math.inf)
    assert not got["dq"][:, 235:].any()
    assert not got["dk"][:, 235:].any() and not got["dv"][:, 235:].any()


@pytest.mark.parametrize("d,dtype", [(64, BF), (80, FP), (96, BF), (128, FP)])
@pytest.mark.parametrize("mask", ["none", "causal", "spans", "packed"])
def test_masks_with_many_workgroups(mask, d, dtype):
    """More rows than the form for few takes with a mask, in numbers of heads that the dies
    share differently."""
    B, H, n = {"none": (2, 100, 200), "causal": (1, 170, 200), "spans": (2, 84, 210),
               "packed": (1, 203, 190)}[mask]
    spans = None
    if mask == "spans":
        spans = _random_spans(41, B, n, n - 9)
    elif mask == "packed":
        spans = torch.zeros(n, 2, dtype=torch.int32)
        for a, b in ((0, 50), (50, 140), (140, n - 11)):
            spans[a:b, 0], spans[a:b, 1] = a, b
        spans = spans.cuda()
    m = n - 9 if mask == "spans" else n
    _compare(*_inputs(42, B, n, m, H, H, d, dtype), spans=spans, causal=mask == "causal")


@pytest.mark.parametrize("bad", [math.nan, math.inf])
def test_masked_places_with_many_workgroups(bad):
    q, k, v, do = _inputs(43, 2, 200, 200, 90, 90, 64, BF)
    spans = torch.zeros(200, 2, dtype=torch.int32)
    spans[:97, 1] = 97
    spans[97:190, 0], spans[97:190, 1] = 97, 190
    for t in (q, k, v, do):
        t[:, 190:] = bad
    _compare(q, k, v, do, spans=spans.cuda())
    q[:, 100] = math.nan  # of the second sequence, in the first one's tile of rows
    tok = _tokens()
    o, lse = tok.attention(q, k, v, spans=spans.cuda())
    nan = torch.isnan(o).any(3).any(2)
    assert torch.equal(nan, torch.arange(200, device="cuda").expand(2, 200) == 100)


def test_rows_that_all_see_nothing():
    q, k, v, do = _inputs(9, 2, 70, 90, 2, 2, 64, BF)
    got = _compare(q, k, v, do, spans=torch.zeros(70, 2, dtype=torch.int32).cuda())
    for n in ("o", "dq", "dk", "dv"):
        assert not got[n].any(), n


@pytest.mark.parametrize("bad", [math.nan, math.inf, -math.inf])
@pytest.mark.parametrize("H,n", [(2, 150), (64, 150), (1, 20)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_what_masked_places_hold_reaches_nothing(bad, H, n, dtype):
    """A packed row: sequences end inside tiles, and padding holds NaN or infinity."""
    q, k, v, do = _inputs(10, 1, n, n, H, H, 64, dtype)
    cut, pad = n // 2 - 3, n - 7
    spans = torch.zeros(n, 2, dtype=torch.int32)
    spans[:cut, 1] = cut
    spans[cut:pad, 0], spans[cut:pad, 1] = cut, pad
    for t in (q, k, v, do):
        t[:, pad:] = bad
    _compare(q, k, v, do, spans=spans.cuda())


@pytest.mark.parametrize("H", [2, 64])
def test_nan_of_one_sequence_stays_in_it(H):
    q, k, v, do = _inputs(11, 1, 140, 140, H, H, 64, BF)
    spans = torch.zeros(140, 2, dtype=torch.int32)
    spans[:75, 1] = 75
    spans[75:, 0], spans[75:, 1] = 75, 140
    v[:, 80] = math.nan
    q[:, 100] = math.nan
    tok = _tokens()
    sp = spans.cuda()
    o, lse = tok.attention(q, k, v, spans=sp)
    g = tok.attention_bwd(do, q, k, v, o, lse, spans=sp)
    clean = [t[:, :75].contiguous() for t in (q, k, v, do)]
    want = ref.attention(*clean[:3], ref.spans_of(75, 75), 0.125, clean[3])
    for n, x in (("o", o), ("dq", g[0]), ("dk", g[1]), ("dv", g[2])):
        ref.check(n, x[:, :75], want[n])
    assert torch.isnan(o[:, 75:]).all() and torch.isnan(g[0][:, 75:]).all()
    assert torch.isnan(g[1][:, 75:]).all()
    assert torch.isnan(g[2][:, 75:]).all()


def test_scores_far_apart_and_reference_moves():
    """Scores grow along the keys, so the running reference moves in every tile; and fall."""
    for sign in (1.0, -1.0):
        q, k, v, do = _inputs(12, 1, 40, 400, 2, 2, 64, BF)
        ramp = torch.linspace(0.1, 6.0, 400)[None, :, None, None].cuda()
        k = (k.float().abs() * ramp * sign).to(BF)
        q = q.abs()
        _compare(q, k, v, do)
        _compare(q.repeat(1, 1, 32, 1), k.repeat(1, 1, 32, 1), v.repeat(1, 1, 32, 1),
                 do.repeat(1, 1, 32, 1))


@pytest.mark.parametrize("H,n", [(64, 700), (2, 700)])
@pytest.mark.parametrize("rise", [0.5, 8.0, 12.0, 40.0])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_scores_that_rise_along_the_keys(H, n, rise, dtype):
    """Each 64 keys' scores pass those before by `rise` powers of two, for every second query;
    the others' fall as fast. The gradients where p spans less than its 32 bits can (2^-126),
    or than its 16 bits beside the largest in fp16; the bounds leave underflow out."""
    q, k, v, do = _inputs(21, 1, n, n, H, H, 64, dtype)
    q[..., 0], k[..., 0] = 1.0, 0.0
    q[:, ::2, :, 0] = -1.0
    step = rise * math.log(2.0) / 64
    k[0, :, :, 0] = (torch.arange(n, device="cuda") * step - n * step / 2)[:, None].to(dtype)
    span = 120 if dtype == BF else 24
    _compare(q, k, v, do if rise * n / 64 < span else None, scale=1.0)


def test_long_row_of_small_probabilities_in_fp16():
    """Probabilities below fp16's normal range (2^-14) keep their precision in the gradient."""
    q, k, v, do = _inputs(13, 1, 33, 20000, 1, 1, 64, FP)
    _compare(q * 0.1, k * 0.1, v, do * 0.01)


@pytest.mark.parametrize("do_scale", [2.0 ** -12, 2.0 ** 8])
def test_gradient_scales_in_fp16(do_scale):
    q, k, v, do = _inputs(14, 1, 150, 150, 2, 2, 64, FP)
    _compare(q, k, v, do * do_scale)


def test_strided_views_broadcasts_and_given_outputs():
    """Views of one joint projection, a key cache with room behind, one batch entry for all."""
    tok = _tokens()
    joint = _randn(15, 2, 100, 4 + 2 + 2, 64)
    q, k, v = joint[:, :, :4], joint[:, :, 4:6], joint[:, :, 6:]
    do = _randn(16, 2, 4, 100, 64).transpose(1, 2)
    _compare(q, k, v, do)
    cache = _randn(17, 3, 500, 2, 64)
    _compare(q, cache[:2, 17:317], cache[1:, 40:340], do)
    one = cache[:1, :90].expand(2, -1, -1, -1)
    _compare(q, one, one, do)
    out = torch.full((2, 100, 6, 64), 7.0, dtype=BF, device="cuda")
    o, _ = tok.attention(q, k, v, out=out[:, :, 1:5])
    assert torch.equal(o, tok.attention(q, k, v)[0])
    assert torch.all(out[:, :, 0] == 7) and torch.all(out[:, :, 5] == 7)


def test_no_keys_and_no_queries():
    tok = _tokens()
    q, k, v, do = _inputs(18, 2, 5, 0, 2, 2, 64, BF)
    o, lse = tok.attention(q, k, v)
    assert not o.any() and torch.all(lse == -math.inf)
    dq, dk, dv = tok.attention_bwd(do, q, k, v, o, lse)
    assert not dq.any() and dk.numel() == 0
    q, k, v, do = _inputs(19, 2, 0, 5, 2, 2, 64, BF)
    o, lse = tok.attention(q, k, v)
    dq, dk, dv = tok.attention_bwd(do, q, k, v, o, lse)
    assert o.numel() == 0 and not dk.any() and not dv.any()


def test_splits_agree_with_one_pass():
    """A long cache for a few rows (parts joined) against the same rows among many."""
    tok = _tokens()
    q, k, v, _ = _inputs(20, 1, 160, 9000, 8, 4, 128, BF)
    few, few_lse = tok.attention(q[:, :2], k, v)
    many = q.repeat(1, 8, 1, 1)
    full, full_lse = tok.attention(many, k, v)
    want = ref.attention(q[:, :2], k, v, ref.spans_of(2, 9000), 1 / math.sqrt(128))
    ref.check("o", few, want["o"])
    ref.check("lse", few_lse, want["lse"])
    ref.check("o", full[:, :2], want["o"])
    ref.check("lse", full_lse[:, :, :2], want["lse"])


def test_nan_in_a_row_shows_in_parts_too():
    """A NaN query, a NaN key and a NaN value in a long cache that is computed in parts."""
    tok = _tokens()
    q, k, v, _ = _inputs(31, 1, 3, 9000, 2, 2, 64, BF)
    q[:, 1] = math.nan
    v[:, 5000, 1, 7] = math.nan
    o, lse = tok.attention(q, k, v)
    assert torch.isnan(o[:, 1]).all() and torch.isnan(lse[:, :, 1]).all()
    assert torch.isfinite(o[:, 0, 0]).all() and torch.isfinite(lse[:, :, 0]).all()
    assert torch.isnan(o[:, 0, 1, 7]) and int(torch.isnan(o[:, 0, 1]).sum()) == 1
    k[:, 8999, 0, 3] = math.nan
    o, lse = tok.attention(q, k, v)
    assert torch.isnan(o[:, 0, 0]).all() and torch.isnan(lse[:, 0]).all()


def test_offsets_past_32_bits():
    """A cache of more than 2^32 bytes (2^31 elements); the queries see its end."""
    n, d = 2_200_000, 128
    cache = torch.empty(1, n, 8, d, dtype=BF, device="cuda")
    cache[:, -300:] = _randn(21, 1, 300, 8, d)
    q, do = _randn(22, 1, 40, 4, d), _randn(23, 1, 40, 4, d)
    k, v = cache[:, :, :4], cache[:, :, 4:]
    spans = torch.tensor([[n - 300, n]] * 40, dtype=torch.int32).cuda()
    tok = _tokens()
    o, lse = tok.attention(q, k, v, spans=spans)
    dq, dk, dv = tok.attention_bwd(do, q, k, v, o, lse, spans=spans)
    want = ref.attention(q, k[:, -300:], v[:, -300:], ref.spans_of(40, 300), 1 / math.sqrt(d), do)
    for name, x in (("o", o), ("lse", lse), ("dq", dq), ("dk", dk[:, -300:]), ("dv", dv[:, -300:])):
        ref.check(name, x, want[name])
    assert not dk[:, :-300].any() and not dv[:, :-300].any()


def test_equal_inputs_give_equal_bits():
    tok = _tokens()
    q, k, v, do = _inputs(24, 2, 300, 700, 8, 2, 128, BF)
    runs = []
    for _ in range(3):
        o, lse = tok.attention(q, k, v, causal=True)
        runs.append((o, lse, *tok.attention_bwd(do, q, k, v, o, lse, causal=True)))
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))


def test_on_another_stream():
    tok = _tokens()
    s = torch.cuda.Stream()
    q, k, v, do = _inputs(25, 1, 200, 200, 4, 4, 64, BF)
    s.wait_stream(torch.cuda.current_stream())
    o, lse = tok.attention(q, k, v, stream=s)
    g = tok.attention_bwd(do, q, k, v, o, lse, stream=s)
    s.synchronize()
    want = ref.attention(q, k, v, ref.spans_of(200, 200), 0.125, do)
    for n, x in (("o", o), ("lse", lse), ("dq", g[0]), ("dk", g[1]), ("dv", g[2])):
        ref.check(n, x, want[n])


def test_gradient_against_differences():
    """dL/dx . t against central differences of the 64-bit forward along t."""
    q, k, v, do = _inputs(26, 1, 50, 70, 4, 2, 64, FP)
    spans = _random_spans(27, 1, 50, 70)
    allowed = ref.spans_of(50, 70, spans)
    tok = _tokens()
    o, lse = tok.attention(q, k, v, spans=spans)
    grads = tok.attention_bwd(do, q, k, v, o, lse, spans=spans)
    xs = [t.cpu().double() for t in (q, k, v)]
    g64 = do.cpu().double()

    def loss(xs):
        qq, kk, vv = (x.transpose(1, 2) for x in xs)
        kk, vv = (x.repeat_interleave(2, 1) for x in (kk, vv))
        s = (qq @ kk.transpose(2, 3) * 0.125).masked_fill(~allowed, -math.inf)
        return float((torch.softmax(s, 3).nan_to_num(0.0) @ vv * g64.transpose(1, 2)).sum())

    bounds = ref.attention(q, k, v, allowed, 0.125, do)
    for i, name in enumerate(("dq", "dk", "dv")):
        t = torch.randn(xs[i].shape, generator=torch.Generator().manual_seed(i), dtype=torch.float64)
        h = 1e-5
        up, down = list(xs), list(xs)
        up[i], down[i] = xs[i] + h * t, xs[i] - h * t
        diff = (loss(up) - loss(down)) / (2 * h)
        got = float((grads[i].cpu().double() * t).sum())
        # the element bounds along t, and the differences' own error (h^2 and 64-bit rounding)
        room = float((bounds[name][1] * t.abs()).sum()) + 1e-6 * (1 + abs(diff))
        assert abs(got - diff) <= room, (name, got, diff, room)


def test_autograd_matches_the_calls():
    tok = _tokens()
    q, k, v, do = _inputs(28, 1, 90, 90, 4, 2, 64, BF)
    xs = [t.clone().requires_grad_() for t in (q, k, v)]
    o = tok.Attention.apply(*xs, None, True, None)
    o.backward(do)
    o2, lse = tok.attention(q, k, v, causal=True)
    assert torch.equal(o, o2)
    for x, g in zip(xs, tok.attention_bwd(do, q, k, v, o2, lse, causal=True)):
        assert torch.equal(x.grad, g)


def test_in_a_graph():
    """Captured and replayed on new inputs, with eager work between the replays."""
    tok = _tokens()
    q, k, v, do = _inputs(29, 1, 4, 3000, 8, 2, 128, BF)
    ws = torch.empty(tok.attention_workspace_size(q, k), dtype=torch.uint8, device="cuda")
    out = torch.empty_like(q)
    tok.attention(q, k, v, out=out, workspace=ws)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        _, lse = tok.attention(q, k, v, out=out, workspace=ws)
        grads = tok.attention_bwd(do, q, k, v, out, lse)
    for i in range(4):
        q.copy_(_randn(100 + i, 1, 4, 8, 128))
        g.replay()
        got = [t.clone() for t in (out, lse, *grads)]
        o2, lse2 = tok.attention(q, k, v)
        want = (o2, lse2, *tok.attention_bwd(do, q, k, v, o2, lse2))
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)), i


def test_refusals():
    import gaussian_splatting_differentiable_amd as gsr
    tok = _tokens()
    q, k, v, do = _inputs(30, 1, 8, 8, 4, 2, 64, BF)

    def status(*a, **kw):
        with pytest.raises(gsr.GsError) as e:
            tok.attention(*a, **kw)
        return e.value.status

    assert status(q.float(), k.float(), v.float()) == gsr.GS_ERR_UNSUPPORTED
    assert status(q[..., :60], k[..., :60], v[..., :60]) == gsr.GS_ERR_UNSUPPORTED
    wide = torch.zeros(1, 8, 2, 136, dtype=BF, device="cuda")
    assert status(wide, wide, wide) == gsr.GS_ERR_UNSUPPORTED
    assert status(q[:, :, :3], k, v) == gsr.GS_ERR_INVALID_ARGUMENT
    assert status(q, k, v, scale=-1.0) == gsr.GS_ERR_INVALID_ARGUMENT
    assert status(q, k, v, scale=math.nan) == gsr.GS_ERR_INVALID_ARGUMENT
    flat = torch.zeros(8 * 4 * 64 + 8, dtype=BF, device="cuda")
    odd = flat[4:4 + 8 * 4 * 64].view(1, 8, 4, 64)         # 8 bytes off
    assert status(odd, k, v) == gsr.GS_ERR_INVALID_ARGUMENT
    for bad in (lambda: tok.attention(q, k, v[:, :4]), lambda: tok.attention(q, k.half(), v),
                lambda: tok.attention(q, k, v, spans=torch.zeros(7, 2, dtype=torch.int32).cuda()),
                lambda: tok.attention(q, k, v, spans=torch.zeros(8, 2).cuda()),
                lambda: tok.attention(q.cpu(), k, v), lambda: tok.attention(q[0], k, v),
                lambda: tok.attention(q.transpose(2, 3), k, v),
                lambda: tok.attention_bwd(do[:, :4], q, k, v, q, q)):
        with pytest.raises(ValueError):
            bad()
