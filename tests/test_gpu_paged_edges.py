"""Edges of the paged cache's operators: infinities that a row sees, weights below 16 bits, tiles at
every cut of the split, empty pools, steps of many tokens."""
import math

import pytest
import torch

import ref_paged as ref
from hierarchical_chunk_sparse_scoring_b200 import binding as hb

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def dense_table(lens, page):
    """A table of consecutive pages for rows of these lengths, and the pages in use."""
    need = [-(-n // page) for n in lens]
    M = max(need) + 1
    at, rows = 0, []
    for c in need:
        rows.append(list(range(at, at + c)) + [-1] * (M - c))
        at += c
    return ints(rows), at


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (8, 1), (16, 1)])
@pytest.mark.parametrize("n", [1, 2, 50, 4000])
def test_attn_infinite_values_that_are_seen(n, Hq, Hkv, dtype):
    """An infinite value reaches the output as itself: a positive weight times it."""
    g = torch.Generator(device="cuda").manual_seed(n)
    d, page = 64, 16
    table, P = dense_table([n], page)
    K, V = [torch.randn((P, Hkv, page, d), generator=g, device="cuda").to(dtype) for _ in range(2)]
    q = torch.randn((1, Hq, d), generator=g, device="cuda").to(dtype)
    if n == 50:
        K.zero_()     # equal weights, exactly one
    want, wlse = hb.paged_attn(q, K, V, table, ints([n - 1]))
    for j, i, v in ((n - 1, 3, math.inf), (0, 5, -math.inf), (n // 2, 63, math.inf)):
        V[j // page, :, j % page, i] = v
    out, lse = hb.paged_attn(q, K, V, table, ints([n - 1]))
    assert bool((out[..., 3] == math.inf).all()) and bool((out[..., 63] == math.inf).all())
    assert bool((out[..., 5] == -math.inf).all())
    rest = [i for i in range(d) if i not in (3, 5, 63)]
    assert torch.equal(out[..., rest], want[..., rest]) and torch.equal(lse, wlse)


@pytest.mark.parametrize("Hq", [1, 4, 16])
def test_attn_weights_keep_32_bits(Hq):
    """Three tokens with values 0, 1 and -1 and logits 0, -x and -x - e: out is a difference of two
    weights that agree in sixteen bits.  u = 2^-24: a logit is exact but for its factor (2 u x, x
    below 0.7), a weight within 2 u more, the sums of products within 12 u, and the division by
    more than two halves that: 8 u."""
    d, page, T, e = 64, 8, 64, 2.0 ** -16
    xs = 0.125 + torch.arange(1, T + 1, dtype=torch.float64) / 128     # (exact in bf16)
    K = torch.zeros((T, 1, page, d), device="cuda")
    V = torch.zeros((T, 1, page, d), device="cuda")
    K[:, 0, 1:3, 0] = -xs.float().cuda()[:, None]
    K[:, 0, 2, 1] = -e
    V[:, 0, 1], V[:, 0, 2] = 1.0, -1.0
    q = torch.zeros((T, Hq, d), device="cuda")
    q[..., :2] = 1.0
    out, _ = hb.paged_attn(q.to(BF), K.to(BF), V.to(BF), ints([[t] for t in range(T)]),
                           ints([2] * T), scale=1.0)
    a, b = torch.exp(-xs), torch.exp(-xs - e)
    want = ((a - b) / (1 + a + b))[:, None, None].expand(T, Hq, d)
    ref.within(out, want, torch.full_like(want, 8 * ref.U), BF)


def test_attn_sums_of_long_rows_have_no_bias():
    """Rows of 65536 tokens, thousands of tiles a warp: sums that are cut off and not rounded to
    nearest would lean to one side with their length.  The values are positive and vary over many
    steps of bf16, so the outputs' own roundings (half a step of 2^-7 at most, 2^-8 / sqrt(3)
    each on average) fall evenly: their mean over N outputs is within 6 2^-8 / sqrt(3 N).  What
    32 bits leave is a few u in each tile and 8 u sqrt(tiles) in rounded sums."""
    T, Hq, d, n, page = 512, 8, 128, 65536, 64
    g = torch.Generator(device="cuda").manual_seed(5)
    K, V = [torch.randn((n // page, 1, page, d), generator=g, device="cuda") for _ in range(2)]
    K, V = K.to(BF), (0.5 + V.abs()).to(BF)
    q = (3 * torch.randn((T, Hq, d), generator=g, device="cuda")).to(BF)
    table = torch.arange(n // page, device="cuda", dtype=torch.int32)[None]
    out, lse = hb.paged_attn(q, K, V, table, ints([n - 1] * T), seq=ints([0] * T))
    off, worst = 0.0, 0.0
    for t in range(0, T, 64):
        x = q[t:t + 64].double().flatten(0, 1) @ K.double().reshape(n, d).T / math.sqrt(d)
        z = torch.logsumexp(x, -1)
        o = torch.exp(x - z[:, None]) @ V.double().reshape(n, d)
        off += float((out[t:t + 64].double().flatten(0, 1) / o - 1).sum())
        worst = max(worst, float((lse[t:t + 64].double().flatten() - z).abs().max()))
    N = T * Hq * d
    print("mean of the relative differences", off / N, "of the lse at most", worst)
    assert abs(off / N) <= 6 * 2.0 ** -8 / math.sqrt(3 * N) + 8 * ref.U * math.sqrt(n / 16)


def test_append_to_an_empty_pool():
    """Padding asks for nothing, so nothing is recorded; a slot that no pool holds is."""
    T, d = 593, 64
    q, k, v = [torch.randn((T, h, d), device="cuda") for h in (2, 1, 1)]
    K = torch.empty((0, 1, 16, d), device="cuda")
    ws = hb.paged_workspace(device="cuda")
    for slots, status in (([-1] * T, 0), ([-1] * (T - 1) + [0], 5)):
        out = torch.full((T, 2, d), 7.0, device="cuda")
        hb.paged_append(q, k, v, None, None, hb.rope(64), K, K.clone(), ints([0] * T), ints(slots),
                        q_out=out, ws=ws)
        assert hb.device_status(ws) == status and bool((out == 7).all())


def test_calls_without_a_workspace_record_where_it_can_be_read():
    hb.paged_status()
    d, page = 64, 16
    g = torch.Generator(device="cuda").manual_seed(1)
    K, V = [torch.randn((4, 1, page, d), generator=g, device="cuda") for _ in range(2)]
    q = torch.randn((2, 2, d), generator=g, device="cuda")
    good, pos = ints([[0, 1], [2, 3]]), ints([20, 30])

    def plan(new):
        return hb.paged_plan(ints([5]), ints([new]), ints([[0, -1]]), ints([3, 2, 1, 0]), ints([2]),
                             page_size=page, T_cap=64)

    def append(slot):
        return hb.paged_append(q, q[:, :1], q[:, :1], None, None, hb.rope(d), K, V, pos, ints(slot))

    def attn(table, rows=q):
        return hb.paged_attn(rows, K, V, table, pos)

    for ok, bad in ((lambda: plan(3), lambda: plan(40)),
                    (lambda: append([-1, 3]), lambda: append([3, 64])),
                    (lambda: attn(good), lambda: attn(ints([[0, 4], [2, 3]])))):
        ok()
        assert hb.paged_status() == 0
        bad()
        ok()
        assert hb.paged_status() == 5 and hb.paged_status() == 0
    # the word survives a workspace that has to grow, and belongs to its stream
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    append([64, 64])
    wide = torch.randn((2, 16, d), generator=g, device="cuda")
    attn(good, wide)
    hb.paged_attn(q, K, V, good, pos, stream=side)
    assert hb.paged_status(side) == 0 and hb.paged_status() == 5
    # a captured call has a workspace of its own
    want = attn(good)
    p = pos.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = hb.paged_attn(q, K, V, good, p)
    p.fill_(1 << 20)
    graph.replay()
    assert hb.paged_status() == 0
    p.copy_(pos)
    graph.replay()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
