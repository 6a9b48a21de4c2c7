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


def split_places(lens, Hkv, kt):
    """Places of the split's list for rows of these lengths: a unit of n tiles takes n + 1."""
    return sum(-(-n // kt) + 1 for n in lens if n) * Hkv


def check_every_tile(lens, Hq, Hkv, dtype, d=64, window=0):
    """With q = 0 every weight is one and lse = ln n; V is one-hot in the group of eight tokens, so
    each group adds one eighth of a tile's count to a dimension of its own (groups 8 d tokens apart
    share one).  Weights, factors and sums are whole numbers below 2^24, exact in 32 bits, so an
    output is a count over n within the division (3 u) and its rounding, and the logarithm within
    4 u of its value."""
    page = 64
    table, P = dense_table(lens, page)
    V = torch.zeros((P, Hkv, page, d), device="cuda", dtype=dtype)
    at = 0
    dims = torch.arange(max(max(lens), 1), device="cuda") // 8 % d
    for n in lens:
        j = torch.arange(n, device="cuda")
        V[at + j // page, :, j % page, dims[:n]] = 1.0
        at += -(-n // page)
    K = torch.zeros_like(V)
    q = torch.zeros((len(lens), Hq, d), device="cuda", dtype=dtype)
    out, lse = hb.paged_attn(q, K, V, table, ints([n - 1 for n in lens]), window=window)
    lo = [max(0, n - window) if window else 0 for n in lens]
    count = torch.zeros((len(lens), d), dtype=torch.float64, device="cuda")
    for t, n in enumerate(lens):
        count[t] = torch.bincount(dims[lo[t]:n], minlength=d)[:d]
    size = torch.tensor([float(n - a) for n, a in zip(lens, lo)], dtype=torch.float64,
                        device="cuda")
    want = torch.where(size[:, None] > 0, count / size.clamp(min=1)[:, None], 0.0)
    got = out.double()
    half = ref.HALF_STEP[dtype]
    assert bool(((got - want[:, None]).abs() <= (half + 3 * ref.U) * want[:, None]).all()), lens
    wl = torch.log(size)
    ok = (lse.double() == wl[:, None]) | ((lse.double() - wl[:, None]).abs() <=
                                          4 * ref.U * (wl[:, None].abs() + 1))
    assert bool(ok.all()), lens


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("lens,Hq,Hkv", [
    ([70001], 8, 1), ([70001], 1, 1), ([30011, 3, 50000], 16, 1), ([20000, 0, 0, 9999], 4, 4),
    ([131072, 131071], 6, 2), ([1] * 500 + [60000] + [2] * 300, 2, 2)])
def test_attn_every_tile_of_long_rows(lens, Hq, Hkv, dtype):
    check_every_tile(lens, Hq, Hkv, dtype)
    check_every_tile(lens, Hq, Hkv, dtype, d=128, window=17003)


@pytest.mark.parametrize("dtype,kt", [(BF, 16), (F32, 8)], ids=["bf16", "fp32"])
def test_attn_every_tile_at_every_cut(dtype, kt):
    """A short row before a long one moves the long one's cuts place by place: over a whole stretch
    of a block and then some, so that blocks and warps begin at a unit's own place, at its first
    tile, behind it, and at the place after a whole stretch."""
    ctas = torch.cuda.get_device_properties(0).multi_processor_count
    base = kt * ctas * 20
    per = split_places([base], 1, kt) // ctas + 1
    seen = set()
    for shift in range(0, per + 12):
        lens = [shift * kt, base, 5 * kt]
        step = max(4, int(split_places(lens, 1, kt) / ctas) + 1)
        seen |= {((c * step) - split_places(lens[:1], 1, kt)) for c in range(ctas)
                 if 0 <= c * step - split_places(lens[:1], 1, kt) <= step + 1}
        check_every_tile(lens, 8, 1, dtype)
    assert {0, 1, 2, per - 1, per, per + 1} <= seen


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hkv", [(8, 1), (16, 1), (4, 4), (6, 2)])
def test_attn_every_tile_of_random_batches(Hq, Hkv, dtype):
    g = torch.Generator().manual_seed(Hq)
    for i in range(40):
        T = int(torch.randint(1, 200, (1,), generator=g))
        top = int(2 ** (4 + 10 * float(torch.rand(1, generator=g))))
        lens = torch.randint(0, top, (T,), generator=g).tolist()
        lens[int(torch.randint(0, T, (1,), generator=g))] = 20 * top
        check_every_tile(lens, Hq, Hkv, dtype, window=[0, 0, 3 * top // 2][i % 3])


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("tokens", [131072, 160001, 400009])
def test_plan_of_many_tokens(tokens, in_place):
    """More tokens than the grid has threads, the last round not a whole one."""
    B, page = 53, 16
    g = torch.Generator().manual_seed(tokens)
    kv = torch.randint(0, 3000, (B,), generator=g)
    new = torch.full((B,), tokens // B)
    new[7] += tokens - int(new.sum()) - 9
    have, end = (kv + page - 1) // page, (kv + new + page - 1) // page
    P, M = int(end.sum()) + 3, int(end.max()) + 1
    perm = torch.randperm(P, generator=g)
    first = have.cumsum(0) - have
    col = torch.arange(M)[None]
    table = torch.where(col < have[:, None], perm[(first[:, None] + col).clamp(max=P - 1)], -1)
    n_free = P - int(have.sum())
    free = torch.cat([perm[int(have.sum()):], torch.zeros(P - n_free, dtype=torch.long)])
    # the pages a sequence takes come from the top of the stack in order of (sequence, page)
    before = (end - have).cumsum(0) - (end - have)
    fresh = (col >= have[:, None]) & (col < end[:, None])
    want = torch.where(fresh, free[(n_free - 1 - (before[:, None] + col - have[:, None])).clamp(
        0, P - 1)], table)
    n = int(new.sum())
    seq = torch.repeat_interleave(torch.arange(B), new)
    cu = torch.cat([torch.zeros(1, dtype=torch.long), new.cumsum(0)])
    pos = kv[seq] + torch.arange(n) - cu[seq]
    tail = torch.full((tokens - n,), -1)
    tab, kvt, nft = ints(table.tolist()), ints(kv.tolist()), ints([n_free])
    kw = dict(kv_len_out=kvt, n_free_out=nft) if in_place else {}
    ws = hb.paged_workspace(device="cuda")
    got = hb.paged_plan(kvt, ints(new.tolist()), tab, ints(free.tolist()), nft, page_size=page,
                        T_cap=tokens, ws=ws, **kw)
    assert hb.device_status(ws) == 0
    assert torch.equal(tab.cpu().long(), want)
    slot = want[seq, pos // page] * page + pos % page
    for name, w in (("seq", seq), ("pos", pos), ("slot", slot)):
        assert torch.equal(got[name].cpu().long(), torch.cat([w, tail])), name
    assert torch.equal(got["cu"].cpu().long(), cu)
    assert torch.equal(got["kv_len"].cpu().long(), kv + new)
    assert got["n_free"].tolist() == [n_free - int((end - have).sum())]


@pytest.mark.parametrize("idle", [1, 31, 32, 33, 64, 1000, 20000])
def test_attn_idle_rows_between_live_ones(idle):
    """Rows without a sequence or without tokens, in runs of every length up to `idle`, between rows
    that see something (a batch whose requests come and go).  The rows' values are those of the
    live rows alone, within what another split may change, and a run costs no read per row: with
    1334 idle rows a step takes less than five times one without them (1.2 times where it was
    measured; a dependent read each would take 0.17 us, a dozen times in all)."""
    g = torch.Generator(device="cuda").manual_seed(idle)
    runs = sorted({0, 1, idle // 3, idle})
    live, seq, pos = [], [], []
    for b, run in enumerate(runs):
        live.append(len(seq))
        seq.append(b)
        pos.append(1500 + 100 * b)
        for i in range(run):
            seq.append([-1, b][i % 2])
            pos.append([700, -1][i % 2])
    live.append(len(seq))
    seq.append(0)
    pos.append(40)
    T, Hq, d, page = len(seq), 8, 128, 64
    K, V = [torch.randn((40 * len(runs), 1, page, d), generator=g, device="cuda").to(BF)
            for _ in range(2)]
    table = torch.arange(40 * len(runs), device="cuda", dtype=torch.int32).view(len(runs), 40)
    q = torch.randn((T, Hq, d), generator=g, device="cuda").to(BF)
    seq, pos, at = ints(seq), ints(pos), torch.tensor(live, device="cuda")
    out, lse = torch.full_like(q, 3.0), torch.full((T, Hq), 3.0, device="cuda")
    ws = hb.paged_workspace(q, K)

    def batch():
        hb.paged_attn(q, K, V, table, pos, seq=seq, out=out, lse=lse, ws=ws)
    alone = [t[at].contiguous() for t in (q, pos, seq)]

    def few():
        return hb.paged_attn(alone[0], K, V, table, alone[1], seq=alone[2], ws=ws)
    batch()
    want, wlse = few()
    assert hb.device_status(ws) == 0
    # each side is within half a step of bf16 and 2^-12 of values that sum |p V| < 8 bounds
    assert bool(((out[at].double() - want.double()).abs() <=
                 2 * 2.0 ** -8 * want.double().abs() + 2.0 ** -12).all())
    assert bool(((lse[at] - wlse).abs() <= 1e-5).all())
    rest = torch.ones(T, dtype=torch.bool, device="cuda")
    rest[at] = False
    pad, empty = rest & (seq < 0), rest & (seq >= 0)
    assert bool((out[pad] == 3).all()) and bool((lse[pad] == 3).all())
    assert bool((out[empty] == 0).all()) and bool((lse[empty] == -math.inf).all())

    def fastest(f):
        times = []
        for _ in range(10):
            a, b = [torch.cuda.Event(enable_timing=True) for _ in range(2)]
            torch.cuda.synchronize()
            a.record()
            for _ in range(5):
                f()
            b.record()
            torch.cuda.synchronize()
            times.append(a.elapsed_time(b))
        return min(times)
    if idle == 1000:
        assert fastest(batch) < 5 * fastest(few)
