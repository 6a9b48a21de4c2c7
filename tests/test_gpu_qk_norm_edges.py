"""Edges of qk_norm_rope's backward: no eps, and weight gradients of many rows."""
import pytest
import torch

import ref_paged as ref
from hierarchical_chunk_sparse_scoring_b200 import binding as hb

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def d64(t):
    return t.double().cpu()


@pytest.mark.parametrize("dtype,grad", [(BF, F32), (BF, BF), (F32, F32)],
                         ids=["bf16-g32", "bf16-g16", "fp32"])
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("B,N,Hq,Hkv,d", [
    (1, 1, 8, 1, 128), (1, 33, 8, 1, 128), (2, 1501, 3, 1, 64), (1, 5003, 4, 2, 64),
    (1, 700, 5, 5, 96), (1, 3, 7, 3, 256)])
def test_weight_gradients_without_eps(B, N, Hq, Hkv, d, layout, dtype, grad):
    """eps = 0 is allowed: odd head counts, tails of tokens and few tokens leave places without a
    row, which have no norm."""
    g = torch.Generator(device="cuda").manual_seed(N)
    q, k = [torch.randn((B, h, N, d), generator=g, device="cuda").to(dtype) for h in (Hq, Hkv)]
    wq, wk = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype) for _ in range(2)]
    dys = [torch.randn(x.shape, generator=g, device="cuda").to(grad) for x in (q, k)]
    rope, (freq, ms) = hb.rope(32, layout=layout), ref.frequencies(32)
    out = hb.qk_norm_rope_backward(q, k, wq, wk, *dys, rope, eps=0.0)
    pos = torch.arange(N)[None].expand(B, N)
    for x, w, dy, n in ((q, wq, dys[0], "q"), (k, wk, dys[1], "k")):
        dx, dw, dx_b, dw_b = ref.norm_rope_backward(d64(x), d64(w), pos, d64(dy), freq, ms, layout,
                                                    eps=0.0)
        ref.within(out["d" + n], dx, dx_b, grad)
        ref.within(out["dw_" + n], dw, dw_b)


@pytest.mark.parametrize("d", [8, 64, 128, 256])
def test_weight_gradients_keep_small_rows(d):
    """Rows whose shares lie below half a step of the sum they are added to are not lost.  With
    x = 1 and eps = 0 a row's share is dy itself, exact; large ones of both signs come first, so
    that every running sum holds one when the small ones arrive.  A token has one head, so no sum
    is held in 32 bits but the last rounding; the product and the norm's root add at most 3 u."""
    N = (1 << 25) // d
    big = 20000
    x = torch.ones((1, 1, N, d), device="cuda")
    dy = torch.full((1, 1, N, d), 2.0 ** -25, device="cuda")
    dy[:, :, :big] = 1.0
    dy[:, :, 1:big:2] = -1.0
    w = torch.ones(d, device="cuda")
    got = hb.qk_norm_rope_backward(x, None, w, None, dy, None, hb.rope(0), eps=0.0)["dw_q"]
    want = (N - big) * 2.0 ** -25
    assert bool(((got.double() - want).abs() <= 5 * ref.U * want).all()), (got[0].item(), want)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,Hq,Hkv,d", [(20011, 1, 1, 16), (20011, 3, 2, 64), (12007, 5, 2, 128),
                                        (9477, 2, 3, 256)])
def test_weight_gradients_of_single_rows(T, Hq, Hkv, d, dtype):
    """Gradients that are zero but for the rows where a walk over the tokens can go wrong: the last
    tokens, the last head, the first tokens of a later round.  A share is a product within 20 u
    (g 6, x r 11, the products) of (|a| + |b|) |x r|, and a token's few heads add one each."""
    g = torch.Generator(device="cuda").manual_seed(T + d)
    q, k = [torch.randn((1, h, T, d), generator=g, device="cuda").to(dtype) for h in (Hq, Hkv)]
    wq, wk = [torch.ones(d, device="cuda").to(dtype) for _ in range(2)]
    rot = min(d, 64)
    rope, (freq, ms) = hb.rope(rot), ref.frequencies(rot)
    rounds = [592 * t for t in (1, 2, 4, 8, 16)]
    spots = [[T - 1], [T - 3, T - 2], [t for t in rounds if t < T], [t - 1 for t in rounds if t <= T],
             [0], list(range(T - T % 16, T))]
    for i, tokens in enumerate(spots):
        dys = []
        for h in (Hq, Hkv):
            dy = torch.zeros((1, h, T, d), device="cuda")
            heads = [h - 1] if i % 2 else list(range(h))
            for t in tokens:
                dy[0, heads, t] = torch.randn((len(heads), d), generator=g, device="cuda")
            dys.append(dy.to(dtype))
        out = hb.qk_norm_rope_backward(q, k, wq, wk, *dys, rope)
        at = torch.tensor(tokens)
        for x, dy, n in ((q, dys[0], "q"), (k, dys[1], "k")):
            xs, ys = d64(x[:, :, at.cuda()]), d64(dy[:, :, at.cuda()])
            p = at.double()[None, None]
            share = ref.turn(ys, p, freq, ms, "half", sign=-1.0) * xs * torch.rsqrt(
                xs.square().mean(-1, keepdim=True) + 1e-6)
            mag = ref._spread(ys, rot, "half") * (xs * torch.rsqrt(
                xs.square().mean(-1, keepdim=True) + 1e-6)).abs()
            ref.within(out["dw_" + n], share.sum((0, 1, 2)), (20 + x.shape[1]) * ref.U *
                       mag.sum((0, 1, 2)))


def test_weight_gradients_past_32_bits():
    """More than 2^31 elements: dw against the sum of two calls over halves of the tokens.  Each is
    one rounding of a sum whose tokens were added in 64 bits, their 32 heads in 32 (40 u of the
    sum of magnitudes with the products)."""
    N, H, d = 530000, 32, 128
    q = torch.empty((1, N, H, d), dtype=BF, device="cuda").normal_(
        generator=torch.Generator(device="cuda").manual_seed(2)).transpose(1, 2)
    w = torch.ones(d, dtype=BF, device="cuda")
    rope = hb.rope(0)
    dw = hb.qk_norm_rope_backward(q, None, w, None, q, None, rope)["dw_q"].double()
    cut = N // 2 + 5
    parts = [hb.qk_norm_rope_backward(q[:, :, a:b], None, w, None, q[:, :, a:b], None,
                                      rope)["dw_q"].double() for a, b in ((0, cut), (cut, N))]
    # the gradients are q itself: shares q^2 r, all positive, so the sum is that of magnitudes
    assert bool(((dw - parts[0] - parts[1]).abs() <= 80 * ref.U * dw).all())
