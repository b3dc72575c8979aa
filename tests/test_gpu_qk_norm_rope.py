"""The norm and rotation of queries and keys and its gradient (gs_qk_norm_rope,
gs_qk_norm_rope_bwd) against the formulas in 64 bits."""
import math

import pytest

torch = pytest.importorskip("torch")

import token_reference as ref

pytestmark = pytest.mark.gpu

TYPES = [torch.float32, torch.bfloat16, torch.float16]


def _tokens():
    from gaussian_splatting_differentiable_amd import tokens
    return tokens


def _randn(seed, *shape, dtype=torch.float32, scale=1.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(shape, generator=g) * scale).to(dtype).cuda()


def _table(rows, rot, seed=5):
    if not rot:
        return None
    a = torch.rand(rows, rot // 2, generator=torch.Generator().manual_seed(seed),
                   dtype=torch.float64) * 2 * math.pi
    return torch.cat([a.cos(), a.sin()], 1).float().cuda()


def _compare(q, k, wq, wk, table, positions, neighbours, eps=1e-6, seed=50):
    tok = _tokens()
    how = dict(cos_sin=table, positions=positions, neighbours=neighbours, eps=eps)
    qo, ko = tok.qk_norm_rope(q, k, wq, wk, **how)
    dq = None if q is None else _randn(seed, *q.shape, dtype=q.dtype)
    dk = None if k is None else _randn(seed + 1, *k.shape, dtype=k.dtype)
    gq, gk, gwq, gwk = tok.qk_norm_rope_bwd(dq, dk, q, k, wq, wk, **how)
    torch.cuda.synchronize()
    x = q if q is not None else k
    pos = positions if positions is not None else torch.arange(x.shape[1])
    for t, w, y, g, dx, dw in ((q, wq, qo, dq, gq, gwq), (k, wk, ko, dk, gk, gwk)):
        if t is None:
            assert y is None and dx is None
            continue
        want = ref.qk_norm_rope(t, w, table, pos, neighbours, eps, g)
        ref.check("y", y, want["y"])
        ref.check("dx", dx, want["dx"])
        assert (dw is None) == (w is None)
        if w is not None:
            ref.check("dw", dw, want["dw"])
    return qo, ko, gq, gk, gwq, gwk


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("neighbours", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (128, 128), (64, 48), (80, 80), (80, 16), (8, 8),
                                   (256, 64), (96, 0), (24, 8), (136, 136)])
def test_head_and_rotation_sizes(dtype, neighbours, d, rot):
    q, k = _randn(1, 2, 19, 5, d, dtype=dtype, scale=2.0), _randn(2, 2, 19, 3, d, dtype=dtype)
    wq, wk = torch.rand(d).cuda() + 0.5, torch.rand(d).cuda() + 0.5
    pos = torch.randint(0, 30, (2, 19), dtype=torch.int32).cuda()
    _compare(q, k, wq, wk, _table(30, rot), pos if rot else None, neighbours)


@pytest.mark.parametrize("B,n,H,Hk", [(1, 1, 1, 1), (1, 1, 16, 2), (3, 1, 4, 4), (1, 1000, 9, 1),
                                      (2, 257, 2, 13), (1, 5000, 4, 4)])
def test_token_and_head_counts(B, n, H, Hk):
    q, k = _randn(3, B, n, H, 64, dtype=torch.bfloat16), _randn(4, B, n, Hk, 64, dtype=torch.bfloat16)
    w = torch.rand(64).cuda() + 0.5
    _compare(q, k, w, w, _table(n, 32), None, False)


def test_joint_projection_views_shared_positions_and_no_weights():
    joint = _randn(6, 2, 40, 4 + 2 + 2, 64, dtype=torch.bfloat16)
    q, k = joint[:, :, :4], joint[:, :, 4:6]
    pos = torch.randint(0, 50, (40,), dtype=torch.int32).cuda()
    _compare(q, k, None, None, _table(50, 64), pos, False)
    _compare(q, k, torch.rand(64).cuda(), None, None, None, False)


def test_queries_or_keys_alone():
    q, w = _randn(7, 2, 33, 3, 128, dtype=torch.float16), torch.rand(128).cuda() + 0.5
    both = _compare(q, q, w, w, _table(33, 128), None, False)
    one = _compare(q, None, w, None, _table(33, 128), None, False)
    two = _compare(None, q, None, w, _table(33, 128), None, False)
    assert torch.equal(both[0], one[0]) and torch.equal(both[1], two[1])
    assert torch.equal(both[4], one[4])


def test_rows_of_zeros_and_of_large_and_tiny_values():
    q = _randn(8, 1, 12, 2, 64)
    q[:, 0] = 0.0
    q[:, 1] *= 1e15
    q[:, 2] *= 1e-15
    _compare(q, q, None, torch.ones(64).cuda(), _table(12, 64), None, True)


def test_positions_outside_the_table_show_as_nan():
    tok = _tokens()
    q = _randn(9, 1, 4, 2, 64, dtype=torch.bfloat16)
    pos = torch.tensor([0, -1, 7, 6], dtype=torch.int32).cuda()
    out, _ = tok.qk_norm_rope(q, None, cos_sin=_table(7, 32), positions=pos)
    assert torch.isnan(out[0, 1:3, :, :32]).all() and torch.isfinite(out[0, [0, 3]]).all()
    assert torch.isfinite(out[0, 1:3, :, 32:]).all()
    g, _, _, _ = tok.qk_norm_rope_bwd(q, None, q, None, cos_sin=_table(7, 32), positions=pos)
    assert torch.isnan(g[0, 1:3]).all() and torch.isfinite(g[0, [0, 3]]).all()


def test_in_place_and_equal_bits():
    tok = _tokens()
    joint = _randn(10, 2, 300, 8, 64, dtype=torch.bfloat16)
    q, k = joint[:, :, :4], joint[:, :, 4:6]
    w, t = torch.rand(64).cuda(), _table(300, 64)
    qo, ko = tok.qk_norm_rope(q, k, w, w, cos_sin=t)
    runs = [tok.qk_norm_rope_bwd(qo, ko, q, k, w, w, cos_sin=t) for _ in range(3)]
    for r in runs[1:]:
        assert all(torch.equal(a, b) for a, b in zip(runs[0], r))
    v = joint[:, :, 6:].clone()
    tok.qk_norm_rope(q, k, w, w, cos_sin=t, q_out=q, k_out=k)
    assert torch.equal(q, qo) and torch.equal(k, ko) and torch.equal(joint[:, :, 6:], v)


def test_gradient_against_differences():
    tok = _tokens()
    q = _randn(11, 1, 6, 2, 40, dtype=torch.float32)
    w, table = torch.rand(40).cuda() + 0.5, _table(6, 24)
    dy = _randn(12, *q.shape)
    g, _, gw, _ = tok.qk_norm_rope_bwd(dy, None, q, None, w, None, cos_sin=table, eps=1e-2)

    def loss(x, w):
        r = 1 / (x.square().mean(3, keepdim=True) + 1e-2).sqrt()
        return float((ref.rotate(x * r * w, table, torch.arange(6), False) * dy.cpu().double()).sum())

    x64, w64 = q.cpu().double(), w.cpu().double()
    gen, h = torch.Generator().manual_seed(0), 1e-5
    t, tw = torch.randn(x64.shape, generator=gen, dtype=torch.float64), \
        torch.randn(40, generator=gen, dtype=torch.float64)
    dx = (loss(x64 + h * t, w64) - loss(x64 - h * t, w64)) / (2 * h)
    dw = (loss(x64, w64 + h * tw) - loss(x64, w64 - h * tw)) / (2 * h)
    # 32-bit results: 2^-18 of the summed magnitudes, and the differences' error
    for got, diff, size in ((g.cpu().double() * t, dx, 1), (gw.cpu().double() * tw, dw, 1)):
        assert abs(float(got.sum()) - diff) <= 2.0 ** -18 * float(got.abs().sum()) + 1e-7, diff


def test_autograd_matches_the_calls():
    tok = _tokens()
    q, k = _randn(13, 1, 9, 4, 64), _randn(14, 1, 9, 2, 64)
    w, t = torch.rand(64).cuda(), _table(9, 64)
    xs = [x.clone().requires_grad_() for x in (q, k, w, w)]
    a, b = tok.QkNormRope.apply(*xs, t, None, False, 1e-6)
    (a.sum() + 2 * b.sum()).backward()
    want = tok.qk_norm_rope_bwd(torch.ones_like(q), torch.full_like(k, 2.0), q, k, w, w, cos_sin=t)
    for x, g in zip(xs, want):
        assert torch.equal(x.grad, g)


def test_no_tokens():
    tok = _tokens()
    q, w = torch.zeros(2, 0, 4, 64, device="cuda"), torch.ones(64, device="cuda")
    a, b = tok.qk_norm_rope(q, q, w, w)
    assert a.shape == q.shape
    _, _, gw, _ = tok.qk_norm_rope_bwd(a, b, q, q, w, w)
    torch.cuda.synchronize()
    assert not gw.any()


def test_refusals():
    import gaussian_splatting_differentiable_amd as gsr
    tok = _tokens()
    q, t = _randn(15, 1, 8, 2, 64), _table(4, 64)

    def status(*a, **kw):
        with pytest.raises(gsr.GsError) as e:
            tok.qk_norm_rope(*a, **kw)
        return e.value.status

    bad = torch.zeros(1, 8, 2, 60, device="cuda")
    assert status(bad, bad) == gsr.GS_ERR_UNSUPPORTED
    assert status(q, q, cos_sin=_table(8, 12)) == gsr.GS_ERR_UNSUPPORTED
    assert status(q, q, cos_sin=_table(8, 72)) == gsr.GS_ERR_INVALID_ARGUMENT
    assert status(q, q, cos_sin=t) == gsr.GS_ERR_INVALID_ARGUMENT       # fewer rows than tokens
    assert status(q, q, eps=-1.0) == gsr.GS_ERR_INVALID_ARGUMENT
    for f in (lambda: tok.qk_norm_rope(q, q.half()), lambda: tok.qk_norm_rope(None, None),
              lambda: tok.qk_norm_rope(q, q, torch.ones(32, device="cuda")),
              lambda: tok.qk_norm_rope(q, q, cos_sin=t.double()),
              lambda: tok.qk_norm_rope(q, q, cos_sin=t, positions=torch.zeros(8).cuda()),
              lambda: tok.qk_norm_rope(q.long(), q.long())):
        with pytest.raises(ValueError):
            f()
