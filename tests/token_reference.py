"""The token operators' formulas in 64 bits, and how far a kernel may be from them.

Bounds hold element by element and follow from the roundings the kernels make:
every value stored in a 16-bit type, and the probabilities and score gradients
that enter a matrix product as 16-bit operands, are off by at most u relative
(half a unit in the last place: 2^-8 for bfloat16, 2^-11 for float16), plus half
the smallest subnormal for float16. SLACK covers the 32-bit arithmetic between.
"""
import math

import torch

U = {t: torch.finfo(t).eps / 2 for t in (torch.bfloat16, torch.float16, torch.float32)}
TINY = {torch.bfloat16: 0.0, torch.float16: 2.0 ** -25, torch.float32: 0.0}
SLACK = 1.25      # second-order terms and 32-bit sums, against the first-order bound
ULP32 = 2.0 ** -18  # 64 roundings of 32-bit values, relative to the sums of magnitudes


def spans_of(nq, nk, spans=None, causal=False):
    """Allowed pairs [.., nq, nk] from a span list [.., nq, 2] and the causal rule."""
    j = torch.arange(nk)
    ok = torch.ones(nq, nk, dtype=torch.bool)
    if causal:
        ok = ok & (j <= torch.arange(nq)[:, None] + nk - nq)
    if spans is not None:
        s = spans.cpu().long()
        ok = ok & (j >= s[..., :1]) & (j < s[..., 1:])
    return ok


def attention(q, k, v, allowed, scale, do=None):
    """Results and bounds, as a dict name -> (value, bound), in 64 bits on the CPU.

    Masked rows and columns are taken out by selection, so what they hold does
    not matter. q [B, nq, H, d], k, v [B, nk, Hk, d]; allowed [nq, nk] or [B, nq, nk]."""
    dt = q.dtype
    u, tiny = U[dt], TINY[dt]
    share = q.shape[2] // k.shape[2]
    q64, k64, v64 = (t.detach().cpu().double().transpose(1, 2) for t in (q, k, v))
    B, H, nq, d = q64.shape
    nk = k64.shape[2]
    allowed = allowed.expand(B, nq, nk)[:, None]
    used_q, used_k = allowed.any(3)[..., None], allowed.any(2)[..., None]
    zero = torch.zeros((), dtype=torch.float64)
    q64 = torch.where(used_q, q64, zero)
    k64, v64 = (torch.where(used_k, t, zero).repeat_interleave(share, 1) for t in (k64, v64))
    s = (q64 @ k64.transpose(2, 3)) * scale
    s = s.masked_fill(~allowed, -math.inf)
    lse = torch.logsumexp(s, 3)
    p = torch.where(allowed, torch.exp(s - torch.where(lse == -math.inf, zero, lse)[..., None]),
                    zero)
    o = p @ v64
    # error of a score in 32 bits, as a relative error of its probability
    err_s = (q64.abs() @ k64.abs().transpose(2, 3)) * scale * ULP32 + ULP32
    err_s = torch.where(allowed, err_s, zero)
    rel_p = err_s + (p * err_s).sum(3, keepdim=True)
    near = (rel_p * p) @ v64.abs()
    out = {"o": (o, SLACK * (u * (p @ v64.abs()) + near + u * o.abs()) + tiny
                 + tiny * (allowed.double() @ v64.abs())),
           "lse": (lse, SLACK * ((p * err_s).sum(3) + ULP32 * (1 + lse.abs().nan_to_num(0, 0, 0))))}
    if do is not None:
        g = torch.where(used_q, do.detach().cpu().double().transpose(1, 2), zero)
        dp = g @ v64.transpose(2, 3)
        delta = (g * o).sum(3, keepdim=True)
        ds = p * (dp - delta)
        # D comes from the stored o
        err_o = out["o"][1]
        err_delta = (g.abs() * err_o).sum(3, keepdim=True) + ULP32 * (g * o).abs().sum(3, keepdim=True)
        err_dp = ULP32 * (g.abs() @ v64.abs().transpose(2, 3))
        err_ds = u * ds.abs() + p * (err_delta + err_dp) + rel_p * ds.abs()
        dv, dk, dq = p.transpose(2, 3) @ g, ds.transpose(2, 3) @ q64 * scale, ds @ k64 * scale
        b_dv = (p * (u + rel_p)).transpose(2, 3) @ g.abs()
        b_dk = err_ds.transpose(2, 3) @ q64.abs() * scale
        b_dq = err_ds @ k64.abs() * scale
        dv, dk, b_dv, b_dk = (t.unflatten(1, (H // share, share)).sum(2)
                              for t in (dv, dk, b_dv, b_dk))
        for n, x, b in (("dq", dq, b_dq), ("dk", dk, b_dk), ("dv", dv, b_dv)):
            out[n] = (x, SLACK * (b + u * x.abs()) + tiny)
    return {n: (x, b) if n == "lse" else (x.transpose(1, 2), b.transpose(1, 2))
            for n, (x, b) in out.items()}


def check(name, got, want):
    """got (device) within the bound of want = (value, bound); infinities equal."""
    x, b = want
    g = got.detach().cpu().double()
    assert g.shape == x.shape, (name, g.shape, x.shape)
    inf = torch.isinf(x)
    assert torch.equal(g[inf], x[inf]), name
    assert bool(torch.isfinite(g[~inf]).all()), f"{name}: not finite where it should be"
    over = (g - x).abs()[~inf] - b[~inf]
    if over.numel() and float(over.max()) > 0:
        i = int(over.argmax())
        raise AssertionError(f"{name}: off by {float((g - x).abs()[~inf][i]):.3e} where "
                             f"{float(b[~inf][i]):.3e} is allowed; {int((over > 0).sum())} of "
                             f"{over.numel()} over")


def rotate(z, table, positions, neighbours, back=False):
    """R z (R^T z with back) of [B, n, H, d] by a [rows, rot] table."""
    if table is None:
        return z
    half = table.shape[1] // 2
    cs = table.cpu().double()[positions.cpu().long()]
    cs = cs[:, None] if cs.dim() == 2 else cs[:, :, None]
    c, s = cs[..., :half], cs[..., half:] * (-1 if back else 1)
    z = z.clone()
    a, b = ((z[..., 0:2 * half:2].clone(), z[..., 1:2 * half:2].clone()) if neighbours
            else (z[..., :half].clone(), z[..., half:2 * half].clone()))
    x, y = a * c - b * s, a * s + b * c
    if neighbours:
        z[..., 0:2 * half:2], z[..., 1:2 * half:2] = x, y
    else:
        z[..., :half], z[..., half:2 * half] = x, y
    return z


def qk_norm_rope(x, w, table, positions, neighbours, eps, dy=None):
    """name -> (value, bound): y, and dx and dw from dy."""
    u, tiny = U[x.dtype], TINY[x.dtype]
    x64 = x.detach().cpu().double()
    w64 = torch.ones(x.shape[3], dtype=torch.float64) if w is None else w.cpu().double()
    r = 1 / (x64.square().mean(3, keepdim=True) + eps).sqrt()
    y = rotate(x64 * r * w64, table, positions, neighbours)
    # each value is a sum of two products of magnitude at most that of its pair
    size = (x64 * r * w64).abs().amax(3, keepdim=True)
    out = {"y": (y, SLACK * u * y.abs() + ULP32 * size + tiny)}
    if dy is not None:
        g = rotate(dy.detach().cpu().double(), table, positions, neighbours, back=True)
        h, xh = g * w64, x64 * r
        m = (h * xh).mean(3, keepdim=True)
        dx = r * (h - xh * m)
        mag = r * (h.abs().amax(3, keepdim=True) + xh.abs() * (h * xh).abs().mean(3, keepdim=True))
        out["dx"] = (dx, SLACK * u * dx.abs() + ULP32 * mag + tiny)
        gm = g.abs().amax(3, keepdim=True)
        out["dw"] = ((g * xh).sum((0, 1, 2)), ULP32 * (gm * xh.abs()).sum((0, 1, 2)))
    return out


def philox(n, seed, offset):
    """n words of the generator as Python integers, block after block."""
    out = []
    for i in range((n + 3) // 4):
        ctr = (offset + i) % 2 ** 64
        c = [ctr % 2 ** 32, ctr >> 32, 0, 0]
        k = [seed % 2 ** 32, (seed >> 32) % 2 ** 32]
        for _ in range(10):
            m0, m1 = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57
            c = [(m1 >> 32) ^ c[1] ^ k[0], m1 % 2 ** 32, (m0 >> 32) ^ c[3] ^ k[1], m0 % 2 ** 32]
            k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
        out += c
    return out[:n]
