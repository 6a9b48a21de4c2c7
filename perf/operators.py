"""Workloads of the query/key prologue and of the paged cache, and their plain forms.

Five operators that surround the sparse attention when a model is trained or served:

  norm_rope   RMS norm of every query and key head with the rotary position code, one pass
  norm_rope_backward   its gradients (inputs and norm weights)
  plan        block tables, slot map and positions of a step, from the requests' lengths
  append      norm_rope of a step's tokens, keys and values written to their cache slots
  attn        attention of one new token per row over the paged cache

`run` computes them with elementary torch operations, or, where `own` is true, with the
framework's kernels.  `exact` is the definition in 64 bits.
"""
import math
import random

import torch

own = False

_DT = {"bf16": torch.bfloat16, "f32": torch.float32}
_EPS = 1e-6


# ------------------------------------------------------------------------------------ the cases

def listed():
    return [
        # -- norm_rope: a prefill of a 32/8-head model, its q and k slices of one fused projection
        dict(name="norm_rope_prefill", op="norm_rope", dtype="bf16", B=1, N=32768, Hq=32, Hkv=8,
             d=128, rot=128, layout="half", scaling="plain", base=10000.0, fused=True, pos0=0),
        # a small fp32 model: odd length, interleaved pairs on half the head, stretched context,
        # heads-first tensors
        dict(name="norm_rope_f32_partial", op="norm_rope", dtype="f32", B=3, N=1021, Hq=16,
             Hkv=16, d=64, rot=32, layout="interleaved", scaling="yarn", base=10000.0,
             fused=False, pos0=4093),
        # -- norm_rope_backward: the training step; gradients arrive in fp32 from the attention's
        # backward pass
        dict(name="norm_rope_bwd_train", op="norm_rope_backward", dtype="bf16", grad="f32", B=2,
             N=8192, Hq=32, Hkv=8, d=128, rot=128, layout="half", scaling="hope",
             base=10000.0, fused=True, pos0=0),
        dict(name="norm_rope_bwd_small", op="norm_rope_backward", dtype="bf16", grad="bf16", B=1,
             N=517, Hq=16, Hkv=16, d=64, rot=64, layout="interleaved", scaling="linear",
             base=10000.0, fused=False, pos0=0),
        # -- plan: one decode step of a full batch; and a step that mixes prompts and decodes
        dict(name="plan_decode", op="plan", B=256, page=64, max_pages=2048, lo=1, hi=100000,
             new_lo=1, new_hi=1, T_cap=256, lens=11),
        dict(name="plan_mixed", op="plan", B=53, page=16, max_pages=4096, lo=0, hi=30000,
             new_lo=0, new_hi=4400, T_cap=131072, lens=12),
        # -- append: a decode step, and a prompt chunk with a padded tail
        dict(name="append_decode", op="append", dtype="bf16", T=64, pad=0, Hq=32, Hkv=8, d=128,
             rot=128, layout="half", scaling="yarn", base=500000.0, page=64, lens=21),
        dict(name="append_prompt", op="append", dtype="bf16", T=16301, pad=83, Hq=32, Hkv=8,
             d=128, rot=64, layout="half", scaling="ntk", base=10000.0, page=16, lens=22),
        # -- attn: one short request (latency), the ordinary ragged batch, a few long requests,
        # and an fp32 model with a local window
        dict(name="attn_one_short", op="attn", dtype="bf16", T=1, Hq=8, Hkv=1, d=128, page=128,
             lo=1000, hi=1100, window=0, lens=31),
        dict(name="attn_batch", op="attn", dtype="bf16", T=64, Hq=32, Hkv=8, d=128, page=64,
             lo=500, hi=16000, window=0, lens=32),
        dict(name="attn_long", op="attn", dtype="bf16", T=8, Hq=32, Hkv=8, d=128, page=64,
             lo=100000, hi=131072, window=0, lens=33),
        dict(name="attn_f32_window", op="attn", dtype="f32", T=37, Hq=16, Hkv=16, d=64, page=16,
             lo=0, hi=9000, window=2048, lens=34),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _heads(rng):
    return rng.choice([(32, 8), (8, 1), (16, 16), (2, 2), (8, 2), (4, 4), (16, 1), (6, 2), (32, 32)])


def _rotary(rng, d):
    return dict(rot=rng.choice([r for r in (16, 32, 48, 64, 96, 128) if r <= d]),
                layout=rng.choice(["half", "interleaved"]),
                scaling=rng.choice(["plain", "linear", "ntk", "yarn", "hope"]),
                base=rng.choice([10000.0, 500000.0]))


def draw(rng):
    op = rng.choice(["norm_rope", "norm_rope_backward", "plan", "append", "attn", "attn"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    Hq, Hkv = _heads(rng)
    if op in ("norm_rope", "norm_rope_backward"):
        d = rng.choice([64, 96, 128])
        B = rng.choice([1, 1, 2, 3])
        N = max(1, _log(rng, 1, 4_000_000 // (Hq + Hkv) // d // B * 32))
        c = dict(op=op, dtype=dtype, B=B, N=N, Hq=Hq, Hkv=Hkv, d=d, fused=rng.random() < 0.5,
                 pos0=rng.choice([0, 1, _log(rng, 1, 1 << 22)]), **_rotary(rng, d))
        if op == "norm_rope_backward":
            c["N"] = max(1, N // 2)
            c["grad"] = "f32" if dtype == "f32" else rng.choice(["bf16", "f32"])
        return c
    if op == "plan":
        B = _log(rng, 1, 1024)
        page = rng.choice([8, 16, 24, 32, 64, 128])
        new_hi = max(1, _log(rng, 1, 131072 // B + 1))
        return dict(op=op, B=B, page=page, max_pages=_log(rng, 16000, 100000) // page + 9000 // page + 1,
                    lo=0, hi=_log(rng, 10, 15000), new_lo=rng.choice([0, 1]),
                    new_hi=min(new_hi, 8000), T_cap=min(new_hi, 8000) * B + rng.choice([0, 0, 37]),
                    lens=rng.randrange(1 << 30))
    d = rng.choice([64, 128])
    page = rng.choice([8, 16, 24, 64, 128])
    if op == "append":
        T = _log(rng, 1, 300_000_000 // (Hq + 2 * Hkv) // d // 8)
        return dict(op=op, dtype=dtype, T=min(T, 16384), pad=rng.choice([0, 0, 1, 29]), Hq=Hq,
                    Hkv=Hkv, d=d, page=page, lens=rng.randrange(1 << 30), **_rotary(rng, d))
    T = _log(rng, 1, 256)
    most = 1_000_000_000 // (T * Hkv * d * (2 if dtype == "bf16" else 4))
    hi = _log(rng, 2, max(3, min(131072, most)))
    return dict(op=op, dtype=dtype, T=T, Hq=Hq, Hkv=Hkv, d=d, page=page,
                lo=rng.choice([0, 1, hi // 2, hi]), hi=hi,
                window=rng.choice([0, 0, 0, _log(rng, 1, 4096)]), lens=rng.randrange(1 << 30))


def _lengths(c, n):
    """Cache lengths of n requests: spread over lo..hi, evenly on their logarithm."""
    r = random.Random(c["lens"])
    lo, hi = c["lo"], c["hi"]
    return [min(hi, max(lo, _log(r, lo + 1, hi + 1) - 1)) for _ in range(n)]


def _new_lengths(c):
    r = random.Random(c["lens"] + 1)
    return [r.randint(c["new_lo"], c["new_hi"]) for _ in range(c["B"])]


def _rot_args(c):
    """Rotary parameters by name: stretched contexts are 8 times the trained 4096 positions."""
    a = dict(layout=c["layout"], scaling=c["scaling"], base=c["base"])
    if c["scaling"] in ("linear", "ntk", "yarn"):
        a["factor"] = 8.0
    if c["scaling"] in ("yarn", "hope"):
        a["train_len"] = 4096.0
    return a


def work(case):
    c = case
    if c["op"] in ("norm_rope", "norm_rope_backward"):
        es = 2 if c["dtype"] == "bf16" else 4
        el = c["B"] * c["N"] * (c["Hq"] + c["Hkv"]) * c["d"]
        if c["op"] == "norm_rope":
            return {"bytes": 2 * el * es, "flops": 8 * el}
        gs = 2 if c["grad"] == "bf16" else 4
        return {"bytes": el * (es + 2 * gs), "flops": 16 * el}
    if c["op"] == "plan":
        ps, lens, new = c["page"], _lengths(c, c["B"]), _new_lengths(c)
        pages = sum(-(-(l + n) // ps) - -(-l // ps) for l, n in zip(lens, new))
        # lengths in and out, the new pages' ids read and entered, three words a token
        return {"bytes": 4 * (4 * c["B"] + 2 * pages + 3 * c["T_cap"]), "flops": 0}
    es = 2 if c["dtype"] == "bf16" else 4
    if c["op"] == "append":
        el = c["T"] * (c["Hq"] + c["Hkv"]) * c["d"]
        return {"bytes": 2 * el * es + 2 * c["T"] * c["Hkv"] * c["d"] * es, "flops": 8 * el}
    keys = sum(min(l, c["window"]) if c["window"] else l for l in _lengths(c, c["T"]))
    rows = c["T"] * c["Hq"]
    return {"bytes": keys * c["Hkv"] * 2 * c["d"] * es + rows * (2 * c["d"] * es + 4),
            "flops": 4 * keys * c["Hq"] * c["d"]}


# ----------------------------------------------------------------------------------- the inputs

def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _qk(c, g, B, N, extra=0):
    """q, k (and v) as [B, H, N, d]: slices of one fused projection [B, N, H, d], or tensors of
    their own."""
    Hq, Hkv, d, dt = c["Hq"], c["Hkv"], c["d"], _DT[c["dtype"]]
    if c.get("fused", True):
        x = torch.randn((B, N, Hq + (1 + extra) * Hkv, d), generator=g, device="cuda").to(dt)
        x = x.transpose(1, 2)
        return [x[:, :Hq], x[:, Hq:Hq + Hkv]] + ([x[:, Hq + Hkv:]] if extra else [])
    return [torch.randn((B, h, N, d), generator=g, device="cuda").to(dt) for h in (Hq, Hkv)]


def _pages(T, per_row, g, spare):
    """A block table [T, per_row] of distinct pages in a shuffled pool."""
    n = T * per_row + spare
    perm = torch.randperm(n, generator=g, device="cuda").to(torch.int32)
    return perm[:T * per_row].reshape(T, per_row).contiguous(), n


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"c": c}
    op = c["op"]
    if own:
        from hierarchical_chunk_sparse_scoring_b200 import binding as hb
        s["hb"] = hb
        if "rot" in c:
            s["rope"] = hb.rope(c["rot"], **_rot_args(c))
    if op in ("norm_rope", "norm_rope_backward", "append"):
        dt = _DT[c["dtype"]]
        s["w_q"] = (1 + 0.2 * torch.randn(c["d"], generator=g, device="cuda")).to(dt)
        s["w_k"] = (1 + 0.2 * torch.randn(c["d"], generator=g, device="cuda")).to(dt)
    if op in ("norm_rope", "norm_rope_backward"):
        s["q"], s["k"] = _qk(c, g, c["B"], c["N"])
        # documents packed into the row: positions start again after a random length
        cut = int(torch.randint(1, c["N"] + 1, (1,), generator=g, device="cuda"))
        p = torch.arange(c["N"], device="cuda")
        p = torch.where(p < cut, p, p - cut) + c["pos0"]
        s["pos"] = p.to(torch.int32).expand(c["B"], c["N"]).contiguous()
        if op == "norm_rope_backward":
            gt = _DT[c["grad"]]
            s["dy_q"], s["dy_k"] = [torch.randn((c["B"], h, c["N"], c["d"]), generator=g,
                                                device="cuda").to(gt)
                                    for h in (c["Hq"], c["Hkv"])]
    elif op == "plan":
        B, ps, M = c["B"], c["page"], c["max_pages"]
        lens, new = _lengths(c, B), _new_lengths(c)
        have = [-(-l // ps) for l in lens]
        need = sum(-(-(l + n) // ps) - h for l, n, h in zip(lens, new, have))
        P = sum(have) + need + 7
        perm = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
        table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
        first = torch.tensor([0] + have, device="cuda").cumsum(0)[:-1, None]
        col = torch.arange(M, device="cuda")[None]
        used = col < torch.tensor(have, device="cuda")[:, None]
        table[used] = perm[(first + col)[used]]
        s["kv_len"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        s["new_len"] = torch.tensor(new, dtype=torch.int32, device="cuda")
        s["table"], s["free"] = table, torch.zeros(P, dtype=torch.int32, device="cuda")
        s["free"][:P - sum(have)] = perm[sum(have):]
        s["n_free"] = torch.tensor([P - sum(have)], dtype=torch.int32, device="cuda")
    elif op == "append":
        T, n, ps = c["T"] + c["pad"], c["T"], c["page"]
        q, k, v = _qk(c, g, 1, T, extra=1)
        s["q"], s["k"], s["v"] = [x[0].transpose(0, 1) for x in (q, k, v)]     # [T, H, d]
        P = -(-n // ps) + 3
        # where the step's tokens go: runs of slots in a shuffled pool, the padding nowhere
        order = torch.randperm(P, generator=g, device="cuda")
        t = torch.arange(n, device="cuda")
        s["slot"] = torch.full((T,), -1, dtype=torch.int32, device="cuda")
        s["slot"][:n] = (order[t // ps] * ps + t % ps).to(torch.int32)
        s["pos"] = torch.full((T,), -1, dtype=torch.int32, device="cuda")
        s["pos"][:n] = torch.randint(0, 200000, (n,), generator=g, device="cuda").to(torch.int32)
        s["K"], s["V"] = [torch.randn((P, c["Hkv"], ps, c["d"]), generator=g,
                                      device="cuda").to(_DT[c["dtype"]]) for _ in range(2)]
        s["q_out"] = torch.zeros((T, c["Hq"], c["d"]), dtype=_DT[c["dtype"]], device="cuda")
    else:
        T, ps, dt = c["T"], c["page"], _DT[c["dtype"]]
        lens = _lengths(c, T)
        per_row = max(1, -(-max(lens) // ps))
        s["table"], P = _pages(T, per_row, g, 2)
        s["K"], s["V"] = [torch.empty((P, c["Hkv"], ps, c["d"]), dtype=dt, device="cuda").normal_(
            generator=g) for _ in range(2)]
        s["q"] = torch.randn((T, c["Hq"], c["d"]), generator=g, device="cuda").to(dt)
        s["pos"] = torch.tensor(lens, dtype=torch.int32, device="cuda") - 1
    if own and op in ("plan", "append"):
        s["ws"] = hb.paged_workspace(device="cuda")
    if own and op == "attn":
        s["ws"] = hb.paged_workspace(s["q"], s["K"])
    return s


# -------------------------------------------------------------------------------- the plain form

def _frequencies(c):
    rot, base = c["rot"], c["base"]
    a = _rot_args(c)
    m = torch.arange(rot // 2, dtype=torch.float64, device="cuda")
    if c["scaling"] == "ntk":
        base = base * a["factor"] ** (rot / (rot - 2))
    th = base ** (-2.0 * m / rot)
    if c["scaling"] == "linear":
        th = th / a["factor"]
    elif c["scaling"] == "yarn":
        turns = a["train_len"] * th / (2 * math.pi)
        keep = ((turns - 1.0) / (32.0 - 1.0)).clamp(0, 1)
        th = keep * th + (1 - keep) * th / a["factor"]
    elif c["scaling"] == "hope":
        th = torch.where(2 * math.pi / th <= a["train_len"], th, torch.zeros_like(th))
    return th, (0.1 * math.log(a["factor"]) + 1.0 if c["scaling"] == "yarn" else 1.0)


def _angles(c, pos):
    """cos and sin [..., rot/2] of the positions, angles in 64 bits."""
    th, amp = _frequencies(c)
    ang = pos.to(torch.float64)[..., None] * th
    return (torch.cos(ang) * amp).float(), (torch.sin(ang) * amp).float()


def _turn(c, x, cos, sin):
    """Rotates the first rot dimensions of x [..., d] (fp32)."""
    rot = c["rot"]
    y = x.clone()
    if c["layout"] == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2] = a * cos - b * sin
        y[..., rot // 2:rot] = a * sin + b * cos
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2] = a * cos - b * sin
        y[..., 1:rot:2] = a * sin + b * cos
    return y


def _norm(x):
    x = x.float()
    return x, torch.rsqrt((x * x).mean(-1, keepdim=True) + _EPS)


def _plain_norm_rope(c, x, w, cos, sin):
    x, r = _norm(x)
    return _turn(c, x * r * w.float(), cos, sin)


def _plain_backward(c, x, w, dy, cos, sin):
    g = _turn(c, dy.float(), cos, -sin)
    x, r = _norm(x)
    gx = g * x * r
    dw = gx.sum((0, 1, 2), dtype=torch.float64).float()
    h = g * w.float()
    dx = r * (h - x * r * r * (h * x).mean(-1, keepdim=True))
    return dx, dw


def _plain_plan(s):
    c = s["c"]
    ps, T, B = c["page"], c["T_cap"], c["B"]
    old, new = s["kv_len"].long(), s["new_len"].long()
    have = (old + ps - 1) // ps
    need = (old + new + ps - 1) // ps - have
    cu = torch.cat([new.new_zeros(1), new.cumsum(0)])
    cup = need.cumsum(0) - need
    t = torch.arange(T, device="cuda")
    seq = (t[:, None] >= cu[None, 1:]).sum(1)
    ok = seq < B
    seq = torch.where(ok, seq, 0)
    pos = old[seq] + t - cu[seq]
    n_free = s["n_free"].long()
    col = torch.arange(c["max_pages"], device="cuda")[None]
    fresh = (col >= have[:, None]) & (col < (have + need)[:, None])
    at = (n_free - 1 - (cup[:, None] + col - have[:, None])).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], s["table"])
    slot = table[seq, torch.where(ok, pos // ps, 0)].long() * ps + pos % ps
    put = lambda v: torch.where(ok, v, -1).int()
    return {"slot": put(slot), "pos": put(pos), "seq": put(seq), "cu": cu.int(),
            "kv_len": (old + new).int(), "n_free": (n_free - need.sum()).int(), "table": table}


def _plain_append(s):
    c = s["c"]
    ps, dt = c["page"], _DT[c["dtype"]]
    live = s["slot"] >= 0
    cos, sin = [x[:, None] for x in _angles(c, s["pos"])]
    q = _plain_norm_rope(c, s["q"], s["w_q"], cos, sin).to(dt)
    k = _plain_norm_rope(c, s["k"], s["w_k"], cos, sin).to(dt)
    s["q_out"][live] = q[live]
    slot = s["slot"][live].long()
    s["K"][slot // ps, :, slot % ps] = k[live]
    s["V"][slot // ps, :, slot % ps] = s["v"][live]
    return s["q_out"], s["K"], s["V"]


def _plain_attn(s):
    c = s["c"]
    T, Hq, Hkv, d, ps = c["T"], c["Hq"], c["Hkv"], c["d"], c["page"]
    L = s["table"].shape[1] * ps
    j = torch.arange(L, device="cuda")
    out, lse = torch.empty_like(s["q"]), torch.empty((T, Hq), device="cuda")
    for t in range(T):
        pages = s["table"][t].long()
        K = s["K"][pages].transpose(0, 1).reshape(Hkv, L, d).float()
        V = s["V"][pages].transpose(0, 1).reshape(Hkv, L, d).float()
        q = s["q"][t].reshape(Hkv, Hq // Hkv, d).float()
        x = torch.matmul(q, K.transpose(1, 2)) / math.sqrt(d)
        pos = s["pos"][t].long()
        see = j <= pos
        if c["window"]:
            see = see & (j > pos - c["window"])
        x = torch.where(see, x, -math.inf)
        m = x.amax(-1, keepdim=True)
        m0 = torch.where(m == -math.inf, 0.0, m)
        e = torch.exp(x - m0)
        z = e.sum(-1, keepdim=True)
        V = torch.where(see[:, None], V, 0.0)
        o = torch.matmul(e, V) / torch.where(z == 0, 1.0, z)
        out[t] = o.reshape(Hq, d).to(out.dtype)
        lse[t] = (m0 + torch.log(z)).reshape(Hq)
    return out, lse


def run(state):
    s, c = state, state["c"]
    op = c["op"]
    if own:
        hb = s["hb"]
        if op == "norm_rope":
            return hb.qk_norm_rope(s["q"], s["k"], s["w_q"], s["w_k"], s["rope"], pos=s["pos"],
                                   eps=_EPS)
        if op == "norm_rope_backward":
            g = hb.qk_norm_rope_backward(s["q"], s["k"], s["w_q"], s["w_k"], s["dy_q"], s["dy_k"],
                                         s["rope"], pos=s["pos"], eps=_EPS)
            return g["dq"], g["dk"], g["dw_q"], g["dw_k"]
        if op == "plan":
            p = hb.paged_plan(s["kv_len"], s["new_len"], s["table"], s["free"], s["n_free"],
                              page_size=c["page"], T_cap=c["T_cap"], ws=s["ws"])
            return {"slot": p["slot"], "pos": p["pos"], "seq": p["seq"], "cu": p["cu"],
                    "kv_len": p["kv_len"], "n_free": p["n_free"], "table": s["table"]}
        if op == "append":
            q = hb.paged_append(s["q"], s["k"], s["v"], s["w_q"], s["w_k"], s["rope"], s["K"],
                                s["V"], s["pos"], s["slot"], eps=_EPS, q_out=s["q_out"],
                                ws=s["ws"])
            return q, s["K"], s["V"]
        return hb.paged_attn(s["q"], s["K"], s["V"], s["table"], s["pos"], window=c["window"],
                             ws=s["ws"])
    if op == "norm_rope":
        cos, sin = [x[:, None] for x in _angles(c, s["pos"])]
        return tuple(_plain_norm_rope(c, s[n], s["w_" + n], cos, sin).to(_DT[c["dtype"]])
                     for n in ("q", "k"))
    if op == "norm_rope_backward":
        cos, sin = [x[:, None] for x in _angles(c, s["pos"])]
        r = [_plain_backward(c, s[n], s["w_" + n], s["dy_" + n], cos, sin) for n in ("q", "k")]
        gt = _DT[c["grad"]]
        return r[0][0].to(gt), r[1][0].to(gt), r[0][1], r[1][1]
    if op == "plan":
        return _plain_plan(s)
    if op == "append":
        return _plain_append(s)
    return _plain_attn(s)


# ----------------------------------------------------------------------- the definition, 64 bits

def _exact_phase(c, pos):
    """e^(i angle) [..., d/2 or fewer pairs], complex 128."""
    rot, a = c["rot"], _rot_args(c)
    amp = 1.0
    out = []
    for m in range(rot // 2):
        th = math.exp(-2.0 * m / rot * math.log(c["base"]))
        if c["scaling"] == "linear":
            th /= a["factor"]
        elif c["scaling"] == "ntk":
            th = math.exp(-2.0 * m / rot * (math.log(c["base"]) +
                                            rot / (rot - 2.0) * math.log(a["factor"])))
        elif c["scaling"] == "yarn":
            amp = 0.1 * math.log(a["factor"]) + 1.0
            k = min(1.0, max(0.0, (a["train_len"] * th / (2 * math.pi) - 1.0) / 31.0))
            th = th * (k + (1.0 - k) / a["factor"])
        elif c["scaling"] == "hope" and 2 * math.pi / th > a["train_len"]:
            th = 0.0
        out.append(th)
    ang = pos.double()[..., None] * torch.tensor(out, dtype=torch.float64, device="cuda")
    return torch.polar(torch.full_like(ang, amp), ang)


def _exact_turn(c, x, phase):
    rot = c["rot"]
    z = x[..., :rot]
    if c["layout"] == "half":
        z = torch.complex(z[..., :rot // 2], z[..., rot // 2:]) * phase
        z = torch.cat([z.real, z.imag], -1)
    else:
        z = torch.view_as_real(torch.complex(z[..., 0::2], z[..., 1::2]) * phase).flatten(-2)
    return torch.cat([z, x[..., rot:]], -1)


def _exact_rows(c, x, w, phase):
    x = x.double()
    return _exact_turn(c, x * w.double() / torch.sqrt(x.square().mean(-1, keepdim=True) + _EPS),
                       phase)


def _exact_grads(c, x, w, dy, phase):
    """One head at a time: y = R(w x / n), n = sqrt(mean x^2 + eps)."""
    dxs, dw = [], 0
    for h in range(x.shape[1]):
        xh = x[:, h].double()
        g = _exact_turn(c, dy[:, h].double(), phase.conj())
        n = torch.sqrt(xh.square().mean(-1, keepdim=True) + _EPS)
        dw = dw + (g * xh / n).sum((0, 1))
        gw = g * w.double()
        dxs.append(gw / n - xh * (gw * xh).sum(-1, keepdim=True) / (x.shape[-1] * n ** 3))
    return torch.stack(dxs, 1), dw


def exact(case, seed):
    c = case
    s = prepare(case, seed)
    op = c["op"]
    if op == "plan":
        return None                     # whole numbers: nothing is rounded
    if op == "norm_rope":
        ph = _exact_phase(c, s["pos"])
        return tuple(torch.stack([_exact_rows(c, s[n][:, h], s["w_" + n], ph)
                                  for h in range(s[n].shape[1])], 1) for n in ("q", "k"))
    if op == "norm_rope_backward":
        ph = _exact_phase(c, s["pos"])
        (dq, wq), (dk, wk) = [_exact_grads(c, s[n], s["w_" + n], s["dy_" + n], ph)
                              for n in ("q", "k")]
        return dq, dk, wq, wk
    if op == "append":
        n, ps = c["T"], c["page"]
        ph = _exact_phase(c, s["pos"][:n])[:, None]
        q, K, V = s["q_out"].double(), s["K"].double(), s["V"].double()
        q[:n] = _exact_rows(c, s["q"][:n], s["w_q"], ph)
        k = _exact_rows(c, s["k"][:n], s["w_k"], ph)
        slot = s["slot"][:n].long()
        for h in range(c["Hkv"]):
            K[torch.div(slot, ps, rounding_mode="floor"), h, slot.remainder(ps)] = k[:, h]
            V[torch.div(slot, ps, rounding_mode="floor"), h, slot.remainder(ps)] = \
                s["v"][:n, h].double()
        return q, K, V
    T, Hq, Hkv, d, ps = c["T"], c["Hq"], c["Hkv"], c["d"], c["page"]
    out = torch.zeros((T, Hq, d), dtype=torch.float64, device="cuda")
    lse = torch.full((T, Hq), -math.inf, dtype=torch.float64, device="cuda")
    for t, n in enumerate(_lengths(c, T)):
        first = max(0, n - c["window"]) if c["window"] else 0
        if n == 0:
            continue
        j = torch.arange(first, n, device="cuda")
        page, off = s["table"][t].long()[j // ps], j % ps
        for g in range(Hkv):
            K, V = s["K"][page, g, off].double(), s["V"][page, g, off].double()
            q = s["q"][t, g * (Hq // Hkv):(g + 1) * (Hq // Hkv)].double()
            x = q @ K.T / math.sqrt(d)
            z = torch.logsumexp(x, -1)
            lse[t, g * (Hq // Hkv):(g + 1) * (Hq // Hkv)] = z
            out[t, g * (Hq // Hkv):(g + 1) * (Hq // Hkv)] = torch.exp(x - z[:, None]) @ V
    return out, lse
