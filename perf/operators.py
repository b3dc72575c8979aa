"""What the token operators are measured on: attention with its gradient, the
norm and rotation of queries and keys with its gradient, and dropout.

The cases stand for a model that predicts Gaussians from the patch tokens of a
scene's views and is trained through the rasterizer: attention over the tokens
of one scene or of several packed ones, a single new token against the tokens
already there, and dropout of residual branches or of the Gaussians' opacities.
`own` selects the plain form in 32 bits or the framework's calls.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


# ---------------------------------------------------------------------- cases

def listed():
    A = dict(op="attention", train=False, batch=1, mask="none", dtype="bf16")
    Q = dict(op="qk", dtype="bf16", pairs="halves", train=False)
    D = dict(op="dropout", dtype="bf16", per_row=False)
    return [
        # one new token of four scenes against the tokens they hold (8 queries share a key head)
        {**A, "name": "attn_token", "batch": 4, "q_len": 1, "kv_len": 16384, "heads": 16,
         "kv_heads": 2, "dim": 128},
        # a small scene: latency counts
        {**A, "name": "attn_small", "q_len": 256, "kv_len": 256, "heads": 8, "kv_heads": 8,
         "dim": 64},
        # all tokens of a scene's views see each other
        {**A, "name": "attn_scene", "batch": 2, "q_len": 8192, "kv_len": 8192, "heads": 16,
         "kv_heads": 16, "dim": 64},
        # scenes of ragged token counts packed into one row, padding at its end, an odd head size
        {**A, "name": "attn_packed", "q_len": 6037, "kv_len": 6037, "heads": 12, "kv_heads": 4,
         "dim": 80, "mask": "packed", "pieces": 5, "dtype": "fp16"},
        # a training step's attention, forward and backward: tokens in order
        {**A, "name": "attn_train_causal", "train": True, "batch": 2, "q_len": 4096,
         "kv_len": 4096, "heads": 16, "kv_heads": 4, "dim": 128, "mask": "causal"},
        # the same where a view's tokens see its own view and the ones before it, ragged
        {**A, "name": "attn_train_views", "train": True, "q_len": 2331, "kv_len": 2331,
         "heads": 8, "kv_heads": 8, "dim": 64, "mask": "views", "pieces": 9, "dtype": "fp16"},
        # the longest scene of the range
        {**A, "name": "attn_train_long", "train": True, "q_len": 16384, "kv_len": 16384,
         "heads": 8, "kv_heads": 2, "dim": 128},
        # the norm and rotation of one new token of four scenes
        {**Q, "name": "qk_token", "batch": 4, "tokens": 1, "heads": 16, "kv_heads": 2, "dim": 128,
         "rot": 128},
        # of a large batch, out of the joint projection's rows
        {**Q, "name": "qk_scene", "batch": 2, "tokens": 32768, "heads": 16, "kv_heads": 4,
         "dim": 128, "rot": 128},
        # a training step's, forward and backward; part of the head is rotated
        {**Q, "name": "qk_train", "batch": 3, "tokens": 5461, "heads": 12, "kv_heads": 12,
         "dim": 64, "rot": 48, "pairs": "neighbours", "train": True},
        # the opacities of the garden-shaped scene's Gaussians, dropped for a sparse-view step
        {**D, "name": "dropout_opacities", "rows": 1535033, "cols": 1, "dtype": "fp32",
         "residual": False},
        # a residual branch of a large batch of tokens, forward and backward
        {**D, "name": "dropout_tokens", "rows": 32768, "cols": 1024, "residual": True},
    ]


def _spread(rng, lo, hi):
    """A whole number of [lo, hi], its logarithm spread evenly."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    kind = rng.choice(["attention", "attention", "token", "qk", "dropout"])
    dtype = rng.choice(["bf16", "fp16"])
    if kind == "token":
        kv = rng.choice([1, 2, 4])
        return dict(op="attention", train=False, batch=rng.randint(1, 8), q_len=rng.randint(1, 4),
                    kv_len=_spread(rng, 1, 32768), heads=kv * rng.choice([1, 2, 3, 8]),
                    kv_heads=kv, dim=8 * rng.randint(4, 16), mask=rng.choice(["none", "causal"]),
                    dtype=dtype)
    if kind == "attention":
        kv = rng.choice([1, 2, 3, 4, 8])
        heads = kv * rng.choice([1, 1, 2, 4])
        heads = max(heads, 4 * kv) if kv < 3 else heads
        train, batch = rng.random() < 0.5, rng.choice([1, 1, 2, 3])
        # no more scores than the largest listed case has
        n = _spread(rng, 16, int(math.sqrt(16384 * 16384 * 8 / (heads * batch))))
        mask = rng.choice(["none", "causal", "packed", "views"])
        c = dict(op="attention", train=train, batch=batch, q_len=n, kv_len=n, heads=heads,
                 kv_heads=kv, dim=8 * rng.randint(4, 16), mask=mask, dtype=dtype)
        if mask in ("packed", "views"):
            c["pieces"] = rng.randint(2, 16)
        elif rng.random() < 0.3:
            c["q_len"] = rng.randint(1, n)
        return c
    if kind == "qk":
        kv = rng.choice([1, 2, 4, 8])
        dim = 8 * rng.randint(4, 16)
        heads, batch = kv * rng.choice([1, 2, 4]), rng.randint(1, 4)
        return dict(op="qk", dtype=rng.choice(["bf16", "fp16", "fp32"]), batch=batch,
                    tokens=_spread(rng, 1, 2 * 32768 * 20 // (batch * (heads + kv) * 2)),
                    heads=heads, kv_heads=kv, dim=dim, rot=8 * rng.randint(0, dim // 8),
                    pairs=rng.choice(["halves", "neighbours"]), train=rng.random() < 0.5)
    cols = rng.choice([1, 3, 64, 333, 1024])
    return dict(op="dropout", dtype=rng.choice(["bf16", "fp16", "fp32"]),
                rows=_spread(rng, 16, 32768 * 512 // cols), cols=cols,
                residual=rng.random() < 0.5, per_row=rng.random() < 0.3)


def _pieces(case):
    """Starts of the case's pieces and its end: uneven, from the case alone."""
    n, k = case["q_len"], case["pieces"]
    w = [1.0 + math.sin(1.7 * i + 0.3 * k) * 0.8 for i in range(k)]
    cuts, at = [0], 0.0
    for x in w[:-1]:
        at += x / sum(w)
        cuts.append(max(cuts[-1], int(n * at)))
    return cuts + [n]


def _spans(case):
    """Each query's keys [lo, hi) as an int32 array [q_len, 2], or None where the mask is none
    or the causal one. Packed: its own piece; the last piece is padding, which sees nothing.
    Views: its own view and the three before it."""
    if case["mask"] not in ("packed", "views"):
        return None
    cuts = _pieces(case)
    spans = np.zeros((case["q_len"], 2), dtype=np.int32)
    for i in range(len(cuts) - 1):
        a, b = cuts[i], cuts[i + 1]
        if case["mask"] == "packed":
            spans[a:b] = (a, b) if i < len(cuts) - 2 else (0, 0)
        else:
            spans[a:b] = (cuts[max(0, i - 3)], b)
    return spans


def _pairs(case):
    """Unmasked (query, key) pairs of one head."""
    s = _spans(case)
    if s is not None:
        return int((s[:, 1] - s[:, 0]).astype(np.int64).sum())
    nq, nk = case["q_len"], case["kv_len"]
    if case["mask"] == "causal":
        return int(np.clip(np.arange(nq, dtype=np.int64) + 1 + nk - nq, 0, nk).sum())
    return nq * nk


def work(case):
    size = DTYPES[case["dtype"]].itemsize
    if case["op"] == "attention":
        q = case["batch"] * case["q_len"] * case["heads"] * case["dim"]
        k = case["batch"] * case["kv_len"] * case["kv_heads"] * case["dim"]
        flops = 4 * case["dim"] * _pairs(case) * case["heads"] * case["batch"]
        # q, k, v, o and the rows' log sums; the gradient reads do and writes dq, dk, dv
        move = (2 * q + 2 * k) * size + 4 * q // case["dim"]
        if case["train"]:
            flops, move = flops * 7 // 2, move + (2 * q + 2 * k) * size
        return {"bytes": move, "flops": flops}
    if case["op"] == "qk":
        x = case["batch"] * case["tokens"] * (case["heads"] + case["kv_heads"]) * case["dim"]
        return {"bytes": x * size * (4 if case["train"] else 2),
                "flops": x * (20 if case["train"] else 8)}
    x = case["rows"] * case["cols"]
    return {"bytes": x * size * ((3 if case["residual"] else 2) + 2), "flops": 4 * x}


# --------------------------------------------------------------------- inputs

def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    dt = DTYPES[case["dtype"]]

    def normal(*shape, scale=1.0):
        return torch.randn(shape, generator=g, device="cuda").mul_(scale).to(dt)

    s = {"case": case}
    if case["op"] == "attention":
        B, n, m, d = case["batch"], case["q_len"], case["kv_len"], case["dim"]
        s["q"] = normal(B, n, case["heads"], d, scale=1.5)
        s["k"] = normal(B, m, case["kv_heads"], d)
        # the values stay where the joint projection left them, beside its keys
        s["v"] = normal(B, m, 2 * case["kv_heads"], d)[:, :, case["kv_heads"]:]
        spans = _spans(case)
        s["spans"] = None if spans is None else torch.from_numpy(spans).cuda()
        if case["train"]:
            s["do"] = normal(B, n, case["heads"], d)
    elif case["op"] == "qk":
        B, n, d, rot = case["batch"], case["tokens"], case["dim"], case["rot"]
        h, hk = case["heads"], case["kv_heads"]
        joint = normal(B, n, h + 2 * hk, d, scale=2.0)
        s["q"], s["k"] = joint[:, :, :h], joint[:, :, h:h + hk]
        s["wq"] = torch.rand(d, generator=g, device="cuda") + 0.5
        s["wk"] = torch.rand(d, generator=g, device="cuda") + 0.5
        if rot:
            freq = 10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)
            angle = torch.arange(n + 64, dtype=torch.float64)[:, None] * freq
            s["table"] = torch.cat([angle.cos(), angle.sin()], 1).float().cuda()
            s["positions"] = torch.randint(0, n + 64, (B, n), generator=g, device="cuda",
                                           dtype=torch.int32)
        else:
            s["table"] = s["positions"] = None
        if case["train"]:
            s["dq"], s["dk"] = normal(B, n, h, d), normal(B, n, hk, d)
    else:
        shape = (case["rows"], case["cols"])
        s["x"] = torch.rand(shape, generator=g, device="cuda").to(dt) if case["cols"] == 1 \
            else normal(*shape)
        s["residual"] = normal(*shape) if case["residual"] else None
        s["dy"] = normal(*shape)
        # a stream for each run and a place in it that passes 32 bits
        s["p"], s["seed"], s["offset"] = 0.1, (seed << 33) * 977 % 2 ** 62 + 11, \
            (seed << 31) % 2 ** 58 + 2 ** 33 + 5
    return s


# -------------------------------------------------------------- the plain form

def _allowed(case, spans, device):
    """Which pairs the mask leaves, [q_len, kv_len], or None for all."""
    nq, nk = case["q_len"], case["kv_len"]
    j = torch.arange(nk, device=device)
    if spans is not None:
        return (j >= spans[:, :1]) & (j < spans[:, 1:])
    if case["mask"] == "causal":
        return j <= torch.arange(nq, device=device)[:, None] + (nk - nq)
    return None


def _plain_attention(s):
    case = s["case"]
    dt, share = DTYPES[case["dtype"]], case["heads"] // case["kv_heads"]
    scale = 1.0 / math.sqrt(case["dim"])
    q = s["q"].float().transpose(1, 2).contiguous()
    k = s["k"].float().transpose(1, 2).repeat_interleave(share, 1)
    v = s["v"].float().transpose(1, 2).repeat_interleave(share, 1)
    p = torch.matmul(q, k.transpose(2, 3).contiguous()).mul_(scale)
    allowed = _allowed(case, s["spans"], q.device)
    if allowed is not None:
        p.masked_fill_(~allowed, -math.inf)
    top = p.amax(3, keepdim=True)
    top = torch.where(top == -math.inf, torch.zeros_like(top), top)
    p.sub_(top).exp_()
    total = p.sum(3, keepdim=True)
    lse = (total.log() + top).squeeze(3)
    p.div_(torch.where(total == 0, torch.ones_like(total), total))
    o = torch.matmul(p, v)
    out = {"o": o.transpose(1, 2).to(dt), "lse": lse}
    if case["train"]:
        do = s["do"].float().transpose(1, 2).contiguous()
        dv = torch.matmul(p.transpose(2, 3).contiguous(), do)
        ds = torch.matmul(do, v.transpose(2, 3).contiguous())
        ds.sub_((do * o).sum(3, keepdim=True)).mul_(p).mul_(scale)
        del p
        dq = torch.matmul(ds, k)
        dk = torch.matmul(ds.transpose(2, 3).contiguous(), q)
        dk, dv = (t.unflatten(1, (case["kv_heads"], share)).sum(2) for t in (dk, dv))
        out |= {n: t.transpose(1, 2).to(dt) for n, t in (("dq", dq), ("dk", dk), ("dv", dv))}
    return out


def _plain_rotate(x, table, positions, neighbours, back):
    if table is None:
        return x
    half = table.shape[1] // 2
    cs = table[positions.long()][:, :, None]
    c, sn = cs[..., :half], cs[..., half:]
    sn = -sn if back else sn
    turned, rest = x[..., :2 * half], x[..., 2 * half:]
    if neighbours:
        a, b = turned[..., 0::2], turned[..., 1::2]
        return torch.cat([torch.stack([a * c - b * sn, a * sn + b * c], -1).flatten(-2), rest], -1)
    a, b = turned[..., :half], turned[..., half:]
    return torch.cat([a * c - b * sn, a * sn + b * c, rest], -1)


def _plain_qk(s):
    case = s["case"]
    dt, nb = DTYPES[case["dtype"]], case["pairs"] == "neighbours"

    def forward(x, w):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        return _plain_rotate(x * r * w, s["table"], s["positions"], nb, False).to(dt)

    def backward(dy, x, w):
        x = x.float()
        r = torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)
        xh = x * r
        gr = _plain_rotate(dy.float(), s["table"], s["positions"], nb, True)
        h = gr * w
        return (r * (h - xh * (h * xh).mean(-1, keepdim=True))).to(dt), (gr * xh).sum((0, 1, 2))

    out = {"q": forward(s["q"], s["wq"]), "k": forward(s["k"], s["wk"])}
    if case["train"]:
        out["dq"], out["dwq"] = backward(s["dq"], s["q"], s["wq"])
        out["dk"], out["dwk"] = backward(s["dk"], s["k"], s["wk"])
    return out


_LOW = 0xFFFFFFFF


def _random_words(n, seed, offset, device):
    """n 32-bit words of the Philox 4x32 generator (10 rounds) as int64: block offset + i / 4
    of the stream `seed` holds words 4 (i / 4) .. + 3."""
    at = torch.arange((n + 3) // 4, dtype=torch.int64, device=device) + offset
    a, b = at & _LOW, (at >> 32) & _LOW
    c, d = torch.zeros_like(a), torch.zeros_like(a)
    k0, k1 = seed & _LOW, (seed >> 32) & _LOW
    for _ in range(10):
        m0, m1 = a * 0xD2511F53, c * 0xCD9E8D57
        a, b, c, d = (((m1 >> 32) & _LOW) ^ b ^ k0, m1 & _LOW,
                      ((m0 >> 32) & _LOW) ^ d ^ k1, m0 & _LOW)
        k0, k1 = (k0 + 0x9E3779B9) & _LOW, (k1 + 0xBB67AE85) & _LOW
    return torch.stack([a, b, c, d], 1).flatten()[:n]


def _plain_dropout(s):
    case, x = s["case"], s["x"]
    n = case["rows"] if case["per_row"] else case["rows"] * case["cols"]
    keep = _random_words(n, s["seed"], s["offset"], x.device) >= round(s["p"] * 2 ** 32)
    keep = keep[:, None] if case["per_row"] else keep.view(x.shape)
    by = 1.0 / (1.0 - s["p"])
    zero = torch.zeros((), device=x.device)
    y = torch.where(keep, x.float() * by, zero)
    if case["residual"]:
        y = y + s["residual"].float()
    return {"y": y.to(x.dtype), "dx": torch.where(keep, s["dy"].float() * by, zero).to(x.dtype)}


# ------------------------------------------------------------------------ run

def _own(s):
    from gaussian_splatting_differentiable_amd import tokens
    case = s["case"]
    if case["op"] == "attention":
        how = dict(spans=s["spans"], causal=case["mask"] == "causal")
        o, lse = tokens.attention(s["q"], s["k"], s["v"], **how)
        out = {"o": o, "lse": lse}
        if case["train"]:
            out["dq"], out["dk"], out["dv"] = tokens.attention_bwd(
                s["do"], s["q"], s["k"], s["v"], o, lse, **how)
        return out
    if case["op"] == "qk":
        how = dict(cos_sin=s["table"], positions=s["positions"],
                   neighbours=case["pairs"] == "neighbours", eps=1e-6)
        q, k = tokens.qk_norm_rope(s["q"], s["k"], s["wq"], s["wk"], **how)
        out = {"q": q, "k": k}
        if case["train"]:
            out["dq"], out["dk"], out["dwq"], out["dwk"] = tokens.qk_norm_rope_bwd(
                s["dq"], s["dk"], s["q"], s["k"], s["wq"], s["wk"], **how)
        return out
    how = dict(per_row=case["per_row"])
    return {"y": tokens.dropout(s["x"], s["p"], s["seed"], s["offset"], residual=s["residual"],
                                **how),
            "dx": tokens.dropout(s["dy"], s["p"], s["seed"], s["offset"], **how)}


def run(state):
    if own:
        return _own(state)
    return {"attention": _plain_attention, "qk": _plain_qk,
            "dropout": _plain_dropout}[state["case"]["op"]](state)


# ---------------------------------------------------- the definition in 64 bits

def _exact_attention(case, s):
    """Row by row of heads: logits, softmax by log sums, and the chain rule in float64."""
    B, H, d = case["batch"], case["heads"], case["dim"]
    share = H // case["kv_heads"]
    q, k, v = (s[n].double().permute(0, 2, 1, 3).contiguous() for n in "qkv")
    do = s["do"].double().permute(0, 2, 1, 3).contiguous() if case["train"] else None
    o, dq = torch.zeros_like(q), torch.zeros_like(q)
    dk, dv = torch.zeros_like(k), torch.zeros_like(v)
    lse = torch.empty(B, H, case["q_len"], dtype=torch.float64, device=q.device)
    key = torch.arange(case["kv_len"], device=q.device).view(1, -1)
    step = max(1, (1 << 27) // case["kv_len"])
    for b in range(B):
        for h in range(H):
            K, V = k[b, h // share], v[b, h // share]
            for i in range(0, case["q_len"], step):
                rows = slice(i, min(i + step, case["q_len"]))
                logit = (q[b, h, rows] @ K.t()) / math.sqrt(d)
                if s["spans"] is not None:
                    logit[(key < s["spans"][rows, :1]) | (key >= s["spans"][rows, 1:])] = -math.inf
                elif case["mask"] == "causal":
                    row = torch.arange(rows.start, rows.stop, device=q.device).view(-1, 1)
                    logit[key > row + case["kv_len"] - case["q_len"]] = -math.inf
                lse[b, h, rows] = torch.logsumexp(logit, 1)
                prob = torch.softmax(logit, 1).nan_to_num_(0.0)
                o[b, h, rows] = prob @ V
                if case["train"]:
                    g = do[b, h, rows]
                    dv[b, h // share] += prob.t() @ g
                    dp = g @ V.t()
                    dl = prob * (dp - (prob * dp).sum(1, keepdim=True)) / math.sqrt(d)
                    dq[b, h, rows] = dl @ K
                    dk[b, h // share] += dl.t() @ q[b, h, rows]
    out = {"o": o.permute(0, 2, 1, 3), "lse": lse}
    if case["train"]:
        out |= {"dq": dq.permute(0, 2, 1, 3), "dk": dk.permute(0, 2, 1, 3),
                "dv": dv.permute(0, 2, 1, 3)}
    return out


def _exact_qk(case, s):
    """The rotation as a complex product, the gradient through the norm's definition."""
    n2 = case["rot"] // 2
    turn = None
    if n2:
        cs = s["table"].double()[s["positions"].long()].unsqueeze(2)
        turn = torch.complex(cs[..., :n2].contiguous(), cs[..., n2:].contiguous())

    def rotate(z, by):
        if by is None:
            return z
        if case["pairs"] == "neighbours":
            w = torch.view_as_complex(z[..., :2 * n2].unflatten(-1, (n2, 2)).contiguous()) * by
            head = torch.view_as_real(w).flatten(-2)
        else:
            w = torch.complex(z[..., :n2].contiguous(), z[..., n2:2 * n2].contiguous()) * by
            head = torch.cat([w.real, w.imag], -1)
        return torch.cat([head, z[..., 2 * n2:]], -1)

    def both(x, w, dy):
        x, w = x.double(), w.double()
        norm = (x.square().sum(-1, keepdim=True) / case["dim"] + 1e-6).sqrt()
        y = rotate(x / norm * w, turn)
        if dy is None:
            return y, None, None
        g = rotate(dy.double(), None if turn is None else turn.conj())
        along = (g * w * x).sum(-1, keepdim=True) / case["dim"]
        return y, g * w / norm - x * along / norm ** 3, (g * x / norm).sum((0, 1, 2))

    yq, dq, dwq = both(s["q"], s["wq"], s.get("dq"))
    yk, dk, dwk = both(s["k"], s["wk"], s.get("dk"))
    out = {"q": yq, "k": yk}
    if case["train"]:
        out |= {"dq": dq, "dwq": dwq, "dk": dk, "dwk": dwk}
    return out


def _exact_dropout(case, s):
    """The generator on the host, in numpy's unsigned words."""
    n = case["rows"] if case["per_row"] else case["rows"] * case["cols"]
    low, up = np.uint64(0xFFFFFFFF), np.uint64(32)
    at = np.arange((n + 3) // 4, dtype=np.uint64) + np.uint64(s["offset"])
    x = [at & low, at >> up, np.zeros_like(at), np.zeros_like(at)]
    k = [s["seed"] % 2 ** 32, (s["seed"] >> 32) % 2 ** 32]
    for _ in range(10):
        m0, m1 = x[0] * np.uint64(0xD2511F53), x[2] * np.uint64(0xCD9E8D57)
        x = [(m1 >> up) ^ x[1] ^ np.uint64(k[0]), m1 & low,
             (m0 >> up) ^ x[3] ^ np.uint64(k[1]), m0 & low]
        k = [(k[0] + 0x9E3779B9) % 2 ** 32, (k[1] + 0xBB67AE85) % 2 ** 32]
    words = np.stack(x, 1).reshape(-1)[:n]
    factor = (words >= np.uint64(round(s["p"] * 2 ** 32))).astype(np.float64) / (1.0 - s["p"])
    factor = torch.from_numpy(factor).cuda()
    factor = factor.view(-1, 1) if case["per_row"] else factor.view(s["x"].shape)
    y, dx = s["x"].double() * factor, s["dy"].double() * factor
    return {"y": y if s["residual"] is None else y + s["residual"].double(), "dx": dx}


def exact(case, seed):
    return {"attention": _exact_attention, "qk": _exact_qk,
            "dropout": _exact_dropout}[case["op"]](case, prepare(case, seed))
