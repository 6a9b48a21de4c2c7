"""qk_norm_rope and its backward against the 64-bit formulas of ref_paged (which derives the
tolerances), through the C ABI."""
import math

import pytest
import torch

import ref_paged as ref
from hierarchical_chunk_sparse_scoring_b200 import binding as hb

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def rope_of(c):
    kw = dict(scaling=c.get("scaling", "plain"), base=c.get("base", 10000.0),
              factor=c.get("factor", 1.0), train_len=c.get("train_len", 0.0))
    return hb.rope(c["rot"], layout=c["layout"], **kw), ref.frequencies(c["rot"], **kw)


def make(shape, order, dtype, g, pad=0):
    """[B, H, N, d]: heads first, tokens first, or a slice with `pad` heads around it."""
    B, H, N, d = shape
    if order == "heads":
        return torch.randn(shape, generator=g, device="cuda").to(dtype)
    x = torch.randn((B, N, H + 2 * pad, d), generator=g, device="cuda").to(dtype)
    return x[:, :, pad:pad + H].transpose(1, 2)


CASES = {
    "train_bf16": dict(B=2, N=150, Hq=32, Hkv=8, d=128, rot=128, layout="half", dtype=BF,
                       order="tokens"),
    "one_token": dict(B=1, N=1, Hq=8, Hkv=1, d=128, rot=64, layout="half", dtype=BF,
                      order="heads"),
    "yarn_f32_d64": dict(B=3, N=77, Hq=4, Hkv=2, d=64, rot=32, layout="interleaved", dtype=F32,
                         order="tokens", scaling="yarn", factor=8.0, train_len=4096.0),
    "hope_bf16_d96": dict(B=1, N=301, Hq=6, Hkv=3, d=96, rot=96, layout="half", dtype=BF,
                          order="heads", scaling="hope", train_len=2000.0),
    "ntk_f32_d256": dict(B=1, N=9, Hq=3, Hkv=1, d=256, rot=48, layout="half", dtype=F32,
                         order="tokens", scaling="ntk", factor=4.0, base=500000.0),
    "linear_bf16_d256": dict(B=2, N=5, Hq=2, Hkv=2, d=256, rot=256, layout="interleaved",
                             dtype=BF, order="heads", scaling="linear", factor=3.0),
    "norot_d8": dict(B=2, N=33, Hq=5, Hkv=5, d=8, rot=0, layout="half", dtype=F32,
                     order="tokens"),
    "d16_many_tokens": dict(B=1, N=20011, Hq=1, Hkv=1, d=16, rot=16, layout="interleaved",
                            dtype=BF, order="heads"),
    "rotate_only": dict(B=2, N=63, Hq=4, Hkv=4, d=128, rot=128, layout="interleaved", dtype=F32,
                        order="heads", norm=False),
    "no_keys": dict(B=1, N=40, Hq=7, Hkv=0, d=64, rot=64, layout="half", dtype=BF,
                    order="tokens"),
    "no_queries": dict(B=1, N=40, Hq=0, Hkv=3, d=64, rot=16, layout="half", dtype=F32,
                       order="heads"),
}


def inputs(c, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    B, N, d, dt = c["B"], c["N"], c["d"], c["dtype"]
    qk = [make((B, h, N, d), c["order"], dt, g, pad=1) if h else None
          for h in (c["Hq"], c["Hkv"])]
    norm = c.get("norm", True)
    ws = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dt) if norm else None
          for _ in qk]
    pos = torch.randint(0, 1 << 22, (B, N), generator=g, device="cuda").to(torch.int32)
    pos[:, 0] = 0
    pos[:, -1] = (1 << 22) + 3
    return qk, ws, pos, norm, g


def d64(t):
    return None if t is None else t.double().cpu()


@pytest.mark.parametrize("name", sorted(CASES))
def test_forward(name):
    c = CASES[name]
    (q, k), (wq, wk), pos, norm, _ = inputs(c)
    rope, (freq, ms) = rope_of(c)
    outs = hb.qk_norm_rope(q, k, wq, wk, rope, pos=pos, norm=norm)
    for x, w, y in ((q, wq, outs[0]), (k, wk, outs[1])):
        if x is None:
            assert y is None
            continue
        r, b = ref.norm_rope(d64(x), d64(w), pos.cpu(), freq, ms, c["layout"], norm=norm)
        assert y.shape == x.shape and y.is_contiguous()
        ref.within(y, r, b, c["dtype"])


@pytest.mark.parametrize("grad", [F32, BF], ids=["g32", "g16"])
@pytest.mark.parametrize("name", sorted(CASES))
def test_backward(name, grad):
    c = CASES[name]
    if grad == BF and c["dtype"] == F32:
        pytest.skip("fp32 inputs have fp32 gradients")
    (q, k), (wq, wk), pos, norm, g = inputs(c, seed=2)
    rope, (freq, ms) = rope_of(c)
    dys = [None if x is None else make(x.shape, "tokens", grad, g) for x in (q, k)]
    out = hb.qk_norm_rope_backward(q, k, wq, wk, dys[0], dys[1], rope, pos=pos, norm=norm)
    again = hb.qk_norm_rope_backward(q, k, wq, wk, dys[0], dys[1], rope, pos=pos, norm=norm)
    for x, w, dy, n in ((q, wq, dys[0], "q"), (k, wk, dys[1], "k")):
        if x is None:
            assert out["d" + n] is None
            if w is not None:
                assert bool((out["dw_" + n] == 0).all())
            continue
        dx, dw, dx_b, dw_b = ref.norm_rope_backward(d64(x), d64(w), pos.cpu(), d64(dy), freq, ms,
                                                    c["layout"], norm=norm)
        assert out["d" + n].dtype == grad
        ref.within(out["d" + n], dx, dx_b, grad)
        if norm:
            assert out["dw_" + n].dtype == F32
            ref.within(out["dw_" + n], dw, dw_b)
        for key in ("d" + n, "dw_" + n):   # no atomics: the same bits
            if out[key] is not None:
                assert torch.equal(out[key], again[key])


def test_gradient_against_differences():
    """The kernel's gradient along a direction against a difference quotient of the definition."""
    c = CASES["yarn_f32_d64"]
    (q, k), (wq, wk), pos, _, g = inputs(c, seed=3)
    rope, (freq, ms) = rope_of(c)
    dy = make(q.shape, "tokens", F32, g)
    out = hb.qk_norm_rope_backward(q, k, wq, wk, dy, torch.zeros_like(k), rope, pos=pos)
    x, w, y = d64(q), d64(wq), d64(dy)
    dx = torch.randn(x.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(5))
    dw = torch.randn(w.shape, dtype=torch.float64, generator=torch.Generator().manual_seed(6))
    loss = lambda h: (ref.norm_rope(x + h * dx, w + h * dw, pos.cpu(), freq, ms,
                                    c["layout"])[0] * y).sum()
    h = 1e-5
    diff = float((loss(h) - loss(-h)) / (2 * h))
    got = float((d64(out["dq"]) * dx).sum() + (d64(out["dw_q"]) * dw).sum())
    _, _, bx, bw = ref.norm_rope_backward(x, w, pos.cpu(), y, freq, ms, c["layout"])
    # the kernel's bound along the direction, and the quotient's own: h^2 times a third
    # derivative of the loss's size, and fp64 rounding of the loss over 2 h
    slack = float((bx * dx.abs()).sum() + (bw * dw.abs()).sum())
    assert abs(got - diff) <= slack + 1e-6 * float((y.abs().sum()))


def test_positions_from_pos0_and_in_place():
    c = CASES["train_bf16"]
    (q, k), (wq, wk), _, _, _ = inputs(c, seed=4)
    rope, _ = rope_of(c)
    pos0 = (1 << 21) + 7
    pos = (pos0 + torch.arange(c["N"], device="cuda")).to(torch.int32).expand(c["B"], -1)
    a = hb.qk_norm_rope(q, k, wq, wk, rope, pos=pos.contiguous())
    b = hb.qk_norm_rope(q, k, wq, wk, rope, pos0=pos0)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    around = q.transpose(1, 2)._base.clone()
    hb.qk_norm_rope(q, k, wq, wk, rope, pos0=pos0, q_out=q, k_out=k)
    assert torch.equal(a[0], q) and torch.equal(a[1], k)
    full = q.transpose(1, 2)._base     # the heads around the slice stay as they were
    assert torch.equal(full[:, :, 0], around[:, :, 0])
    assert torch.equal(full[:, :, -1], around[:, :, -1])


def test_backward_in_place_and_without_weights():
    c = CASES["hope_bf16_d96"]
    (q, k), (wq, _), pos, _, g = inputs(c, seed=5)
    rope, _ = rope_of(c)
    dq, dk = [make(x.shape, "heads", F32, g) for x in (q, k)]
    ones = torch.ones_like(wq)
    a = hb.qk_norm_rope_backward(q, k, wq, ones, dq, dk, rope, pos=pos)
    b = hb.qk_norm_rope_backward(q, k, wq, None, dq, dk, rope, pos=pos, dq=dq, dk=dk)
    assert b["dw_k"] is None and b["dq"] is dq
    assert torch.equal(a["dq"], dq) and torch.equal(a["dk"], dk)
    assert torch.equal(a["dw_q"], b["dw_q"])


def test_matches_hope_rotate():
    """The half layout with the hope rule is hils_hope_rotate's encoding."""
    g = torch.Generator(device="cuda").manual_seed(8)
    x = torch.randn((2, 3, 200, 128), generator=g, device="cuda")
    rope = hb.rope(128, scaling="hope", train_len=65536.0)
    a = hb.hope_rotate(x, rope_base=10000.0, train_len=65536.0, pos0=12345)
    b, _ = hb.qk_norm_rope(x, None, None, None, rope, pos0=12345, norm=False)
    # both within 24 u of (|a| + |b|) of the same value
    assert bool(((a - b).abs() <= 48 * ref.U * 2 * x.abs().amax(-1, keepdim=True)).all())


def test_rows_of_zeros_and_infinities():
    c = CASES["train_bf16"]
    (q, k), (wq, wk), pos, _, _ = inputs(c, seed=6)
    rope, _ = rope_of(c)
    clean = hb.qk_norm_rope(q, k, wq, wk, rope, pos=pos)
    q[0, 1, 2] = 0
    q[1, 3, 4, 5] = math.inf
    q[1, 5, 6, 7] = math.nan
    y, _ = hb.qk_norm_rope(q, k, wq, wk, rope, pos=pos)
    assert bool((y[0, 1, 2] == 0).all())
    assert bool(y[1, 5, 6].isnan().all())
    touched = torch.zeros(q.shape[:3], dtype=torch.bool, device="cuda")
    touched[0, 1, 2] = touched[1, 3, 4] = touched[1, 5, 6] = True
    assert torch.equal(y[~touched], clean[0][~touched])


def test_stream_and_graph():
    c = CASES["train_bf16"]
    (q, k), (wq, wk), pos, _, g = inputs(c, seed=7)
    rope, _ = rope_of(c)
    dq, dk = [make(x.shape, "heads", BF, g) for x in (q, k)]
    want = hb.qk_norm_rope(q, k, wq, wk, rope, pos=pos)
    grads = hb.qk_norm_rope_backward(q, k, wq, wk, dq, dk, rope, pos=pos)
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    got = hb.qk_norm_rope(q, k, wq, wk, rope, pos=pos, stream=s)
    s.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y = hb.qk_norm_rope(q, k, wq, wk, rope, pos=pos)
        b = hb.qk_norm_rope_backward(q, k, wq, wk, dq, dk, rope, pos=pos)
    for _ in range(2):
        for t in (*y, *b.values()):
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y[0], want[0]) and torch.equal(y[1], want[1])
        for n in grads:
            assert torch.equal(b[n], grads[n])


def test_offsets_past_32_bits():
    """More than 2^31 elements: the last tokens as in a short call of their own, both directions."""
    N, H, d = 530000, 32, 128
    assert N * H * d > 2 ** 31
    q = torch.empty((1, N, H, d), dtype=BF, device="cuda").normal_(
        generator=torch.Generator(device="cuda").manual_seed(1)).transpose(1, 2)
    w = torch.ones(d, dtype=BF, device="cuda")
    rope = hb.rope(d, scaling="linear", factor=4.0)
    tail = q[:, :, -7:]
    want, _ = hb.qk_norm_rope(tail, None, w, None, rope, pos0=N - 7)
    got, _ = hb.qk_norm_rope(q, None, w, None, rope)
    assert torch.equal(got[:, :, -7:], want)
    want = hb.qk_norm_rope_backward(tail, None, w, None, got[:, :, -7:], None, rope, pos0=N - 7)
    dq = hb.qk_norm_rope_backward(q, None, w, None, got, None, rope, dq=got)["dq"]
    assert torch.equal(dq[:, :, -7:], want["dq"])


def test_empty():
    rope = hb.rope(64)
    q = torch.empty((2, 4, 0, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    y, k = hb.qk_norm_rope(q, None, w, None, rope)
    assert y.shape == q.shape and k is None
    g = hb.qk_norm_rope_backward(q, None, w, None, q, None, rope)
    assert bool((g["dw_q"] == 0).all())


def test_refusals():
    rope = hb.rope(64)
    q = torch.zeros((1, 2, 4, 64), device="cuda")
    w = torch.ones(64, device="cuda")
    with pytest.raises(TypeError):
        hb.qk_norm_rope(q.half(), None, None, None, rope)
    with pytest.raises(TypeError):
        hb.qk_norm_rope(q, None, w.bfloat16(), None, rope)
    with pytest.raises(ValueError):
        hb.qk_norm_rope(q, None, w[:32], None, rope)
    with pytest.raises(ValueError):
        hb.qk_norm_rope(q.transpose(2, 3), None, None, None, rope)
    with pytest.raises(ValueError):   # overlapping output rows
        hb.qk_norm_rope(q, None, w, None, rope, q_out=q[:, :1].expand(1, 2, 4, 64))
    with pytest.raises(ValueError):
        hb.qk_norm_rope(q, None, w, None, rope, pos=torch.zeros((1, 3), dtype=torch.int32,
                                                                device="cuda"))
    with pytest.raises(hb.HilsError):   # rotation wider than the head
        hb.qk_norm_rope(q[..., :32].contiguous(), None, None, None, rope)
    with pytest.raises(hb.HilsError):   # base not on a 16-byte boundary
        flat = torch.zeros(8 * 64 + 1, device="cuda")
        hb.qk_norm_rope(flat[1:].view(1, 2, 4, 64), None, None, None, rope)
    with pytest.raises(hb.HilsError):   # weights without a norm
        hb.qk_norm_rope(q, None, w, None, rope, norm=False)
    with pytest.raises(ValueError):
        hb.qk_norm_rope(q.cpu(), None, None, None, rope)
