"""Plain 64-bit implementations of the query/key norms with rotary positions and of the paged
cache, on torch float64 CPU tensors, with the error bounds the GPU tests use.

Bounds count roundings.  u = 2^-24 is half a step of fp32; a result rounded to bf16 adds half a
step of bf16, 2^-8 of the value.
"""
import math

import torch

U = 2.0 ** -24
HALF_STEP = {torch.float32: 2.0 ** -24, torch.bfloat16: 2.0 ** -8}


def frequencies(rot, scaling="plain", base=10000.0, factor=1.0, train_len=0.0, beta_fast=32.0,
                beta_slow=1.0):
    """(radians per position of every pair, mscale)."""
    out = []
    for m in range(rot // 2):
        b = base * factor ** (rot / (rot - 2)) if scaling == "ntk" else base
        th = b ** (-2.0 * m / rot)
        if scaling == "linear":
            th /= factor
        elif scaling == "yarn":
            g = (train_len * th / (2 * math.pi) - beta_slow) / (beta_fast - beta_slow)
            g = min(1.0, max(0.0, g))
            th = g * th + (1 - g) * th / factor
        elif scaling == "hope" and 2 * math.pi / th > train_len:
            th = 0.0
        out.append(th)
    return out, (0.1 * math.log(factor) + 1.0 if scaling == "yarn" else 1.0)


def pairs(rot, layout):
    h = rot // 2
    return [(m, m + h) if layout == "half" else (2 * m, 2 * m + 1) for m in range(h)]


def turn(x, pos, freq, mscale, layout, sign=1.0):
    """Rotates x [..., d] at pos (broadcast against x's leading dimensions)."""
    y = x.clone()
    for m, (a, b) in enumerate(pairs(2 * len(freq), layout)):
        t = pos * freq[m]
        c, s = torch.cos(t) * mscale, torch.sin(t) * mscale * sign
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., a] * s + x[..., b] * c
    return y


def _spread(x, rot, layout):
    """|a| + |b| of every element's pair, |a| where it does not turn."""
    y = x.abs().clone()
    for a, b in pairs(rot, layout):
        s = x[..., a].abs() + x[..., b].abs()
        y[..., a], y[..., b] = s, s
    return y


def norm_rope(x, w, pos, freq, mscale, layout, eps=1e-6, norm=True):
    """(y, bound): x [B, H, N, d], pos [B, N].  Bound: the sum of squares has at most 13
    additions on any path (8 in a lane, 5 across lanes), so the norm factor is within 10 u with
    its mean, sum and root; cosine and sine within 4 u (angle, function, mscale); five products
    and sums: 19, taken as 24 u of (|a| + |b|)."""
    p = pos.double()[:, None]
    n = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w if norm else x
    return (turn(n, p, freq, mscale, layout),
            24 * U * max(1.0, abs(mscale)) * _spread(n, 2 * len(freq), layout))


def norm_rope_backward(x, w, pos, dy, freq, mscale, layout, eps=1e-6, norm=True):
    """dx, dw and their bounds.  g is within 6 u of mscale (|a| + |b|); x r within 11 u; a weight
    gradient adds one rounding per row of every partial sum, at most all rows in a row; the dot
    product h.x has the 13 additions of the norm: dx within
    64 u r (|h| + |x| r^2 mean|h x|)."""
    p = pos.double()[:, None]
    g = turn(dy, p, freq, mscale, layout, sign=-1.0)
    gm = max(1.0, abs(mscale)) * _spread(dy, 2 * len(freq), layout)
    if not norm:
        return g, None, 8 * U * gm, None
    r = torch.rsqrt(x.square().mean(-1, keepdim=True) + eps)
    dw = (g * x * r).sum((0, 1, 2))
    rows = x.shape[0] * x.shape[1] * x.shape[2]
    dw_b = (rows + 32) * U * (gm * (x * r).abs()).sum((0, 1, 2))
    h, hm = g * w, gm * w.abs()
    dx = r * (h - x * r * r * (h * x).mean(-1, keepdim=True))
    dx_b = 64 * U * r * (hm + x.abs() * r * r * (hm * x.abs()).mean(-1, keepdim=True))
    return dx, dw, dx_b, dw_b


def attention(q, K, V, lo, hi, scale, weights_dtype):
    """One row: q [Hq, d] over K, V [n, Hkv, d] tokens lo .. hi - 1.  (out, lse, out bound, lse
    bound).  A logit is within (d + 4) u sum|q k| scale, its weight within that, the exponent's
    rounding (2 u |x - m|) and 4 u relative; sums over tokens add at most n/8 + 64 roundings (eight
    warps take the tiles in turn); bf16 carries each weight as two bf16 for the product with V, half
    a step of half a step, 2^-16."""
    Hq, d = q.shape
    n, Hkv, _ = K.shape
    if hi <= lo:
        z = torch.zeros(Hq, d, dtype=torch.float64)
        return z, torch.full((Hq,), -math.inf, dtype=torch.float64), z, torch.zeros(Hq).double()
    Kh, Vh = [t[lo:hi].repeat_interleave(Hq // Hkv, 1) for t in (K, V)]
    x = torch.einsum("hd,nhd->hn", q, Kh) * scale
    mag = torch.einsum("hd,nhd->hn", q.abs(), Kh.abs()) * scale
    lse = torch.logsumexp(x, -1)
    p = torch.exp(x - lse[:, None])
    out = torch.einsum("hn,nhd->hd", p, Vh)
    pv = torch.einsum("hn,nhd->hd", p, Vh.abs())
    far = (x.amax(-1, keepdim=True) - x).clamp(max=80.0)
    e = ((d + 4) * U * mag + 2 * U * far + 4 * U).amax(-1)
    sums = ((hi - lo) / 8 + 64) * U
    rounded = 2.0 ** -16 if weights_dtype == torch.bfloat16 else 0.0
    out_b = (2 * e[:, None] + 2 * sums + rounded) * pv
    return out, lse, out_b, e + sums + 4 * U * lse.abs()


def within(got, ref, bound, dtype=None):
    """|got - ref| <= bound + half a step of dtype; infinities must match."""
    got = got.detach().double().cpu()
    half = HALF_STEP[dtype or torch.float32]
    same = (got == ref) | ((got - ref).abs() <= (bound + half * ref.abs()) * (1 + half))
    assert bool(same.all()), "off by %g where %g is allowed" % (
        float((got - ref).abs()[~same].max()), float((bound + half * ref.abs())[~same].min()))


def plan(kv_len, new_len, table, free, n_free, page, T, n_pages):
    """The step's plan with Python integers.  Returns a dict like binding.paged_plan's, with the
    new table, and whether anything was refused."""
    B, M = len(kv_len), len(table[0]) if table else 0
    table = [list(r) for r in table]
    slot, pos, seq, cu, out, bad = [-1] * T, [-1] * T, [-1] * T, [0], [], False
    if n_free < 0 or n_free > n_pages:
        bad, n_free = True, min(max(n_free, 0), n_pages)
    asked_tok = asked_pages = taken = t = 0
    for b in range(B):
        n, add = kv_len[b], new_len[b]
        if n < 0 or add < 0 or n + add > M * page:
            bad, add = True, 0
        need = -(-(n + add) // page) - -(-n // page) if add > 0 else 0
        asked_tok += add
        asked_pages += need
        if (add and asked_tok > T) or (need and asked_pages > n_free):
            bad, add, need = True, 0, 0
        have = -(-n // page)
        for i in range(need):
            table[b][have + i] = free[n_free - 1 - taken]
            taken += 1
        for i in range(add):
            pg = table[b][(n + i) // page]
            ok = 0 <= pg < n_pages
            bad = bad or not ok
            slot[t], pos[t], seq[t] = (pg * page + (n + i) % page if ok else -1), n + i, b
            t += 1
        out.append(n + add)
        cu.append(t)
    return dict(slot=slot, pos=pos, seq=seq, cu=cu, kv_len=out, n_free=[n_free - taken],
                table=table), bad
