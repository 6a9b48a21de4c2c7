"""The paged cache (paged_plan, paged_append, paged_attn) against plain 64-bit and integer
implementations (ref_paged, which derives the tolerances), through the C ABI."""
import math

import pytest
import torch

import oracle
import parity
import ref_paged as ref
from hierarchical_chunk_sparse_scoring_b200 import binding as hb

pytestmark = pytest.mark.gpu

BF, F32 = torch.bfloat16, torch.float32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def ints(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


# ------------------------------------------------------------------------------------- the plan

def run_plan(kv, new, page, M, n_free, T, P, seed=0, corrupt=None, in_place=False):
    g = torch.Generator().manual_seed(seed)
    perm = torch.randperm(P, generator=g).tolist()
    table, used = [], 0
    for n in kv:
        have = min(max(0, -(-n // page)), M)
        table.append(perm[used:used + have] + [-7] * (M - have))
        used += have
    free = perm[used:] + [-9] * used
    if corrupt:
        corrupt(table)
    want, bad = ref.plan(kv, new, table, free, n_free, page, T, P)
    ws = hb.paged_workspace(device="cuda")
    B = len(kv)
    tab = ints(table).reshape(B, M)
    kvt, nft = ints(kv), ints([n_free])
    kw = dict(kv_len_out=kvt, n_free_out=nft) if in_place else {}
    got = hb.paged_plan(kvt, ints(new), tab, ints(free), nft, page_size=page, T_cap=T, ws=ws,
                        **kw)
    assert hb.device_status(ws) == (5 if bad else 0)
    assert hb.device_status(ws) == 0
    for n in ("slot", "pos", "seq", "cu", "kv_len", "n_free"):
        assert got[n].tolist() == want[n], n
    assert tab.tolist() == want["table"]
    if in_place:
        assert got["kv_len"] is kvt and got["n_free"] is nft
    return want, bad


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("page", [1, 8, 24, 64])
def test_plan_mixed(page, in_place):
    g = torch.Generator().manual_seed(page)
    B = 37
    kv = torch.randint(0, 300, (B,), generator=g).tolist()
    new = torch.randint(0, 90, (B,), generator=g).tolist()
    kv[3], new[3] = 0, 1
    kv[4], new[4] = 2 * page, 1
    kv[5], new[5] = 2 * page, 0
    M = 400 // page + 2
    P = sum(-(-(a + b) // page) for a, b in zip(kv, new)) + 5
    free = P - sum(-(-a // page) for a in kv)
    _, bad = run_plan(kv, new, page, M, free, sum(new) + 11, P, in_place=in_place)
    assert not bad


def test_plan_decode_batch_and_many_sequences():
    B = 3000
    g = torch.Generator().manual_seed(1)
    kv = torch.randint(0, 200, (B,), generator=g).tolist()
    P = sum(-(-(a + 1) // 16) for a in kv)
    free = P - sum(-(-a // 16) for a in kv)
    _, bad = run_plan(kv, [1] * B, 16, 13, free, B, P, in_place=True)
    assert not bad


def test_plan_one_long_prompt():
    # more tokens than one block takes: the whole cluster writes, in place
    _, bad = run_plan([5, 0], [40001, 1], 64, 700, 640, 40010, 641, in_place=True)
    assert not bad


@pytest.mark.parametrize("kv,new,free,T", [
    ([4, 4, 4], [20, 1, 3], 2, 64),          # too few pages for the first; the others fit theirs
    ([8, 8, 7], [1, 1, 1], 1, 64),           # the second is out of pages, the third needs none
    ([0, 0, 0], [5, 6, 2], 9, 10),           # tokens beyond T: the second and, with it, the third
    ([0, -3, 5], [1, 1, -1], 9, 10),         # negative lengths
    ([30, 31, 32], [2, 2, 1], 9, 10),        # a sequence that outgrows its table row
    ([3, 3], [1, 1], 99, 10),                # a free count beyond the pool
    ([8, 8], [1, 1], -2, 10),                # a negative one
    ([0, 0], [0, 0], 3, 10),
    ([2**31 - 1, 1], [2**31 - 1, 1], 4, 4),  # sums beyond 32 bits
])
def test_plan_refuses(kv, new, free, T):
    run_plan(kv, new, 8, 4, free, T, 24)


def test_plan_bad_page_and_empty():
    def corrupt(table):
        table[1][0] = 99
    want, bad = run_plan([4, 4], [1, 1], 8, 4, 5, 4, 16, corrupt=corrupt)
    assert bad and want["slot"][1] == -1
    run_plan([3, 0], [1, 1], 8, 4, 5, 0, 16)      # T_cap 0: everybody is refused
    ws = hb.paged_workspace(device="cuda")
    got = hb.paged_plan(ints([]), ints([]), ints([]).reshape(0, 4), ints([1, 2]), ints([2]),
                        page_size=8, T_cap=3, ws=ws)
    assert got["slot"].tolist() == [-1] * 3 and got["cu"].tolist() == [0]
    assert got["n_free"].tolist() == [2] and hb.device_status(ws) == 0


# ----------------------------------------------------------------------------------- the append

def pool(P, Hkv, page, d, dtype, order, g):
    if order == "heads":
        return torch.randn((P, Hkv, page, d), generator=g, device="cuda").to(dtype)
    return torch.randn((P, page, Hkv, d), generator=g, device="cuda").to(dtype).transpose(1, 2)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("T,Hq,Hkv,d,rot,page,order", [
    (1, 8, 1, 128, 128, 64, "heads"), (77, 6, 2, 64, 32, 24, "tokens"),
    (1500, 4, 4, 96, 96, 1, "heads"), (30, 3, 3, 256, 128, 16, "tokens")])
def test_append(dtype, T, Hq, Hkv, d, rot, page, order):
    g = gen(T)
    x = torch.randn((T, Hq + 2 * Hkv, d), generator=g, device="cuda").to(dtype)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    wq, wk = [(1 + 0.3 * torch.randn(d, generator=g, device="cuda")).to(dtype) for _ in range(2)]
    P = T // page + 4
    K, V = [pool(P, Hkv, page, d, dtype, order, g) for _ in range(2)]
    slot = torch.randperm(P * page, generator=g, device="cuda")[:T].to(torch.int32)
    pos = torch.randint(0, 1 << 20, (T,), generator=g, device="cuda").to(torch.int32)
    if T > 10:
        slot[3] = slot[T - 1] = -1
    q_out = torch.full((T, Hq, d), 7.0, device="cuda").to(dtype)
    K0, V0 = K.clone(), V.clone()
    ws = hb.paged_workspace(device="cuda")
    rope = hb.rope(rot, layout="interleaved")
    got = hb.paged_append(q, k, v, wq, wk, rope, K, V, pos, slot, q_out=q_out, ws=ws)
    assert got is q_out and hb.device_status(ws) == 0
    # the same values as the dense operator, in their places; everything else as it was
    dq, dk = hb.qk_norm_rope(q.transpose(0, 1)[None], k.transpose(0, 1)[None], wq, wk, rope,
                             pos=pos[None].contiguous())
    live = slot >= 0
    want_q = torch.full_like(q_out, 7.0)
    want_q[live] = dq[0].transpose(0, 1)[live]
    s = slot[live].long()
    K0[s // page, :, s % page] = dk[0].transpose(0, 1)[live]
    V0[s // page, :, s % page] = v[live]
    assert torch.equal(q_out, want_q) and torch.equal(K, K0) and torch.equal(V, V0)


def test_append_bad_slot_is_skipped_and_recorded():
    g = gen(3)
    q, k, v = [torch.randn((4, h, 64), generator=g, device="cuda") for h in (2, 1, 1)]
    K, V = [pool(2, 1, 8, 64, F32, "heads", g) for _ in range(2)]
    K0 = K.clone()
    ws = hb.paged_workspace(device="cuda")
    q_out = torch.full((4, 2, 64), 7.0, device="cuda")
    hb.paged_append(q, k, v, None, None, hb.rope(64), K, V, ints([0, 1, 2, 3]),
                    ints([16, 3, 2**31 - 1, -5]), q_out=q_out, ws=ws)
    assert hb.device_status(ws) == 5
    assert bool((q_out[[0, 2, 3]] == 7).all()) and bool((q_out[1] != 7).any())
    assert torch.equal(V[0, 0, 3], v[1, 0])
    K[0, 0, 3] = K0[0, 0, 3]
    assert torch.equal(K, K0)


# -------------------------------------------------------------------------------- the attention

def attn_case(lens, Hq, Hkv, d, page, dtype, order="heads", seed=0, extra=3, stale=math.nan):
    """Rows with these lengths; what no row may see (other pages, tails of pages) holds `stale`."""
    g = gen(seed)
    T = len(lens)
    M = max(1, max(-(-n // page) for n in lens)) + 1
    need = [-(-n // page) for n in lens]
    P = sum(need) + extra
    perm = torch.randperm(P, generator=g, device="cuda").tolist()
    K, V = [pool(P, Hkv, page, d, dtype, order, g) for _ in range(2)]
    table, seen, used = [], torch.zeros((P, page), dtype=torch.bool), 0
    for n, c in zip(lens, need):
        pages = perm[used:used + c]
        used += c
        table.append(pages + [-1] * (M - c))
        for j in range(0, n, page):
            seen[pages[j // page], :min(page, n - j)] = True
    hide = (~seen).cuda()[:, None, :, None]
    K.masked_fill_(hide, stale)
    V.masked_fill_(hide, stale)
    q = (2 * torch.randn((T, Hq, d), generator=g, device="cuda")).to(dtype)
    return q, K, V, ints(table), ints([n - 1 for n in lens])


def check_attn(q, K, V, table, pos, out, lse, window=0, scale=None, seq=None, rows=None):
    page, d = K.shape[2], K.shape[3]
    scale = scale or 1 / math.sqrt(d)
    for t in (range(q.shape[0]) if rows is None else rows):
        s = t if seq is None else int(seq[t])
        n = int(pos[t]) + 1
        lo = max(0, n - window) if window else 0
        j = torch.arange(n, device="cuda")
        pages = table[s].long()[j // page]
        k, v = [x[pages, :, j % page].double().cpu() for x in (K, V)]
        o, l, ob, lb = ref.attention(q[t].double().cpu(), k, v, lo, n, scale, q.dtype)
        ref.within(out[t], o, ob, q.dtype)
        ref.within(lse[t], l, lb)


HEADS = [(1, 1), (2, 2), (6, 2), (4, 1), (8, 1), (16, 1), (32, 8), (14, 2)]


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("Hq,Hkv", HEADS)
def test_attn_heads(Hq, Hkv, d, dtype):
    lens = [0, 1, 15, 16, 17, 64, 65, 333, 1000]
    c = attn_case(lens, Hq, Hkv, d, 16, dtype, seed=Hq * d)
    ws = hb.paged_workspace(c[0], c[1])
    out, lse = hb.paged_attn(*c, ws=ws)
    assert hb.device_status(ws) == 0
    check_attn(*c, out, lse)
    assert bool((out[0] == 0).all()) and bool((lse[0] == -math.inf).all())
    again = hb.paged_attn(*c, ws=ws)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("order", ["heads", "tokens"])
@pytest.mark.parametrize("page", [1, 7, 8, 24, 64, 128, 1000])
def test_attn_pages(page, order, dtype):
    c = attn_case([5, 40, 1, 0, 611, 129], 8, 2, 128, page, dtype, order=order, seed=page,
                  stale=math.inf)
    out, lse = hb.paged_attn(*c)
    check_attn(*c, out, lse)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("window", [1, 2, 16, 17, 100, 5000])
def test_attn_window(window, dtype):
    lens = [0, 1, 16, 18, 100, 101, 700, 3001]
    q, K, V, table, pos = attn_case(lens, 8, 2, 64, 32, dtype, seed=window)
    # what the window leaves behind may hold anything either
    for t, n in enumerate(lens):
        j = torch.arange(max(0, n - window), device="cuda")
        for c in (K, V):
            c[table[t].long()[j // 32], :, j % 32] = math.nan
    out, lse = hb.paged_attn(q, K, V, table, pos, window=window, scale=0.2)
    check_attn(q, K, V, table, pos, out, lse, window=window, scale=0.2)


@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("Hq,Hkv,d,lens", [(8, 1, 128, [70001]), (16, 1, 64, [30011, 3, 50000]),
                                           (4, 4, 128, [20000, 0, 0, 9999]),
                                           (2, 2, 64, [1] * 500 + [6000] + [2] * 300)])
def test_attn_split_rows(Hq, Hkv, d, lens, dtype):
    """Rows cut over many blocks, among many short ones."""
    c = attn_case(lens, Hq, Hkv, d, 64, dtype, seed=len(lens))
    out, lse = hb.paged_attn(*c)
    check_attn(*c, out, lse, rows=list(range(len(lens)))[:3] + [len(lens) - 1] +
               ([500, 501] if len(lens) > 500 else []))
    again = hb.paged_attn(*c)
    assert torch.equal(out, again[0]) and torch.equal(lse, again[1])


def test_attn_rows_name_their_sequences():
    """Several rows of one sequence (each with its own length), padding rows, one sequence
    unused."""
    q, K, V, table, pos = attn_case([300, 50, 80], 8, 2, 128, 16, BF, seed=9)
    seq, pos = ints([0, 0, 2, -1, 0, 2, -1]), ints([299, 10, 79, 5, 0, 40, -1])
    q = (2 * torch.randn((7, 8, 128), generator=gen(1), device="cuda")).to(BF)
    out, lse = torch.full_like(q, 3.0), torch.full((7, 8), 3.0, device="cuda")
    ws = hb.paged_workspace(q, K)
    hb.paged_attn(q, K, V, table, pos, seq=seq, out=out, lse=lse, ws=ws)
    assert hb.device_status(ws) == 0
    check_attn(q, K, V, table, pos, out, lse, seq=seq, rows=[0, 1, 2, 4, 5])
    for t in (3, 6):
        assert bool((out[t] == 3).all()) and bool((lse[t] == 3).all())


def test_attn_bad_values_are_recorded():
    q, K, V, table, pos = attn_case([100, 100, 100, 100], 4, 1, 64, 16, F32, seed=4, stale=0.0)
    want, _ = hb.paged_attn(q, K, V, table, pos)
    ws = hb.paged_workspace(q, K)
    for seq, p, rows in ((ints([0, 9, 2, 3]), pos, [1]),
                         (None, ints([99, 99, 16 * 8, 99]), [2]),
                         (None, ints([99, 99, 99, -2]), [3]),
                         (None, ints([2**31 - 1, 99, 99, 99]), [0])):
        out, lse = hb.paged_attn(q, K, V, table, p, seq=seq, ws=ws)
        assert hb.device_status(ws) == 5
        keep = [t for t in range(4) if t not in rows]   # (split otherwise: other last bits)
        check_attn(q, K, V, table, pos, out, lse, rows=keep)
        assert bool((out[rows] == 0).all()) and bool((lse[rows] == -math.inf).all())
    # a page outside the pool: its 16 tokens count as unseen
    for page in (K.shape[0], -1, 2**31 - 1):
        bad = table.clone()
        bad[2, 3] = page
        out, lse = hb.paged_attn(q, K, V, bad, pos, ws=ws)
        assert hb.device_status(ws) == 5
        j = torch.tensor([i for i in range(100) if i // 16 != 3], device="cuda")
        k, v = [x[table[2].long()[j // 16], :, j % 16].double().cpu() for x in (K, V)]
        o, l, ob, lb = ref.attention(q[2].double().cpu(), k, v, 0, 84, 0.125, F32)
        ref.within(out[2], o, ob)
        ref.within(lse[2], l, lb)
        assert torch.equal(out[[0, 1, 3]], want[[0, 1, 3]])


def test_attn_large_logits_and_values():
    q, K, V, table, pos = attn_case([777, 16], 8, 2, 128, 32, F32, seed=5, stale=0.0)
    # one token far above the rest, and rows whose logits are all very low
    q[0] *= 40
    K[table[1, 0], :, :16] = -3 * q[1].view(2, 4, 128).mean(1)[:, None]
    out, lse = hb.paged_attn(q, K, V, table, pos)
    check_attn(q, K, V, table, pos, out, lse)


def test_attn_stream_and_graph_follow_the_lengths():
    q, K, V, table, pos = attn_case([900, 20, 333, 0], 8, 2, 128, 64, BF, seed=6)
    ws = hb.paged_workspace(q, K)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, lse = hb.paged_attn(q, K, V, table, pos, ws=ws, stream=s)
    s.synchronize()
    check_attn(q, K, V, table, pos, out, lse)
    p = pos.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        o2, l2 = hb.paged_attn(q, K, V, table, p, ws=ws)
    for cut in (0, 100, 18):
        p.copy_((pos - cut).clamp(min=-1))
        graph.replay()
        torch.cuda.synchronize()
        check_attn(q, K, V, table, p, o2, l2)


def test_attn_empty_and_refusals():
    q, K, V, table, pos = attn_case([10, 20], 4, 2, 64, 16, F32, seed=7)
    out, lse = hb.paged_attn(q[:0], K, V, table, pos[:0])
    assert out.shape == (0, 4, 64)
    with pytest.raises(hb.HilsError):   # G = 17
        hb.paged_attn(torch.zeros((2, 34, 64), device="cuda"), K, V, table, pos)
    with pytest.raises(hb.HilsError):   # more rows than sequences
        hb.paged_attn(q, K, V, table[:1].contiguous(), pos)
    with pytest.raises(hb.HilsError):   # a workspace that is too small
        hb.paged_attn(q, K, V, table, pos, ws=torch.zeros(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(TypeError):
        hb.paged_attn(q.bfloat16(), K, V, table, pos)
    with pytest.raises(ValueError):
        hb.paged_attn(q, K, V.transpose(1, 2).contiguous().transpose(1, 2), table, pos)
    with pytest.raises(TypeError):
        hb.paged_attn(q, K, V, table.long(), pos)
    with pytest.raises(hb.HilsError):   # head dim 32
        hb.paged_attn(q[..., :32].contiguous(), K[..., :32].contiguous(),
                      V[..., :32].contiguous(), table, pos)


def test_attn_many_short_rows_and_one_head_rows():
    """More units than blocks, most of one tile, some cut, some empty, rows of other sequences."""
    g = torch.Generator().manual_seed(3)
    lens = torch.randint(0, 40, (700,), generator=g).tolist()
    lens[10] = lens[650] = 5000
    for dtype in (BF, F32):
        c = attn_case(lens, 4, 2, 64, 8, dtype, seed=1)
        out, lse = hb.paged_attn(*c)
        check_attn(*c, out, lse, rows=[0, 1, 9, 10, 11, 300, 649, 650, 651, 699])
        # every row against the batch of itself alone: another split, the same value
        for t in range(0, 700, 97):
            o, z = hb.paged_attn(c[0][t:t + 1].contiguous(), c[1], c[2], c[3][t:t + 1].contiguous(),
                                 c[4][t:t + 1].contiguous())
            check_attn(c[0][t:t + 1], c[1], c[2], c[3][t:t + 1], c[4][t:t + 1], o, z)


def test_attn_of_an_empty_pool_and_table():
    q = torch.randn((3, 4, 64), device="cuda")
    K = torch.empty((0, 2, 16, 64), device="cuda")
    ws = hb.paged_workspace(q, K)
    table = torch.zeros((3, 2), dtype=torch.int32, device="cuda")
    out, lse = hb.paged_attn(q, K, K.clone(), table, ints([-1, 5, 31]), ws=ws)
    assert hb.device_status(ws) == 5
    assert bool((out == 0).all()) and bool((lse == -math.inf).all())
    out, lse = hb.paged_attn(q, K, K.clone(), table[:, :0].contiguous(), ints([-1, -1, -1]), ws=ws)
    assert hb.device_status(ws) == 0 and bool((out == 0).all())


def test_offsets_past_32_bits():
    """Pools of more than 2^31 elements, the pages in use at their far end: append, then read."""
    Hkv, page, d, P = 8, 64, 128, 33000
    assert P * Hkv * page * d > 2 ** 31
    K, V = [torch.empty((P, Hkv, page, d), dtype=BF, device="cuda") for _ in range(2)]
    g = gen(21)
    n = 200
    table = ints([[P - 1, 3, P - 2, P - 3]])
    j = torch.arange(n, device="cuda")
    slot = (table[0].long()[j // page] * page + j % page).to(torch.int32)
    x = torch.randn((n, 32 + 2 * Hkv, d), generator=g, device="cuda").to(BF)
    rope, ws = hb.rope(d), hb.paged_workspace(x[:1, :32], K)
    w = torch.ones(d, dtype=BF, device="cuda")
    q = hb.paged_append(x[:, :32], x[:, 32:40], x[:, 40:], w, w, rope, K, V, j.to(torch.int32),
                        slot, ws=ws)
    pos = ints([n - 1])
    out, lse = hb.paged_attn(q[-1:].contiguous(), K, V, table, pos, ws=ws)
    assert hb.device_status(ws) == 0
    s = slot.long()
    assert torch.equal(V[s // page, :, s % page], x[:, 40:])
    check_attn(q[-1:], K, V, table, pos, out, lse)


def test_two_streams_at_once():
    cases = [attn_case([4000, 9, 700], 8, 2, 128, 64, BF, seed=31),
             attn_case([100] * 40 + [3000], 16, 16, 64, 16, F32, seed=32)]
    want = [hb.paged_attn(*c) for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    wss = [hb.paged_workspace(c[0], c[1]) for c in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(10):
        got += [hb.paged_attn(*c, stream=s, ws=w) for c, s, w in zip(cases, streams, wss)]
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])


def test_one_workspace_serves_calls_in_turn():
    """Plan, append and attention of several shapes on one workspace, one after another."""
    big = attn_case([3000, 40], 16, 1, 128, 64, BF, seed=2)
    ws = hb.paged_workspace(big[0], big[1])
    for c in (big, attn_case([7, 900, 0], 8, 4, 64, 16, F32, seed=3), big):
        out, lse = hb.paged_attn(*c, ws=ws)
        check_attn(*c, out, lse)
        hb.paged_plan(ints([1]), ints([1]), ints([[0]]), ints([1]), ints([1]), page_size=8,
                      T_cap=1, ws=ws)
        assert hb.device_status(ws) == 0


# ----------------------------------------------------------------------------- used together

@pytest.mark.parametrize("dtype", [BF, F32], ids=["bf16", "fp32"])
def test_serving_steps(dtype):
    """Prompts of three requests in one step, then decode steps in one captured graph: every
    step's attention against the definition on all the tokens given so far."""
    g = gen(11)
    Hq, Hkv, d, page, M, P, B = 8, 2, 128, 16, 12, 30, 3
    freq, ms = ref.frequencies(64, "ntk", factor=4.0)
    rope = hb.rope(64, scaling="ntk", factor=4.0)
    wq, wk = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype) for _ in range(2)]
    K, V = [torch.full((P, Hkv, page, d), math.nan, device="cuda").to(dtype) for _ in range(2)]
    table = torch.full((B, M), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(P, generator=g, device="cuda").to(torch.int32)
    n_free, kv = ints([P]), ints([0] * B)
    keys = [[] for _ in range(B)]
    ws = hb.paged_workspace(torch.empty((1, Hq, d), device="cuda", dtype=dtype), K)

    def tokens(T):
        return torch.randn((T, Hq + 2 * Hkv, d), generator=g, device="cuda").to(dtype)

    def step(x, new, T):
        p = hb.paged_plan(kv, new, table, free, n_free, page_size=page, T_cap=T, kv_len_out=kv,
                          n_free_out=n_free, ws=ws)
        q = hb.paged_append(x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], wq, wk, rope, K, V,
                            p["pos"], p["slot"], ws=ws)
        return p, q, hb.paged_attn(q, K, V, table, p["pos"], seq=p["seq"], ws=ws)

    def check(x, new, p, q, out, lse):
        assert hb.device_status(ws) == 0
        t = 0
        for b, n in enumerate(new):
            for _ in range(n):
                i = len(keys[b])
                y, yb = ref.norm_rope(x[t, :Hq].double().cpu()[None, :, None],
                                      wq.double().cpu(), torch.tensor([[i]]), freq, ms, "half")
                ref.within(q[t], y[0, :, 0], yb[0, :, 0], dtype)
                assert p["seq"][t] == b and p["pos"][t] == i
                keys[b].append(int(p["slot"][t]))
                s = torch.tensor(keys[b], device="cuda")
                k, v = [c[s // page, :, s % page].double().cpu() for c in (K, V)]
                o, l, ob, lb = ref.attention(q[t].double().cpu(), k, v, 0, i + 1,
                                             1 / math.sqrt(d), dtype)
                ref.within(out[t], o, ob, dtype)
                ref.within(lse[t], l, lb)
                assert torch.equal(v[-1], x[t, Hq + Hkv:].double().cpu())
                t += 1
        assert sum(len(set(k)) for k in keys) == len(set(sum(keys, [])))   # no slot twice
        assert kv.tolist() == [len(k) for k in keys]

    x = tokens(70)
    p, q, (out, lse) = step(x, ints([20, 0, 47]), 70)
    check(x, [20, 0, 47], p, q, out, lse)
    assert bool((out[67:] == 0).all())
    x, new = tokens(3), ints([1, 1, 1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        p, q, (out, lse) = step(x, new, 3)
    for s, n in enumerate(([1, 1, 1], [1, 0, 1], [0, 0, 0], [1, 1, 0])):
        x.copy_(tokens(3))
        new.copy_(ints(n))
        graph.replay()
        torch.cuda.synchronize()
        check(x, n, p, q, out, lse)


def test_training_chain():
    """qk_norm_rope -> landmarks -> forward -> backward -> its own backward, in fp32, against the
    oracle on the same selection."""
    g = gen(12)
    B, Hq, Hkv, N, d, S, K_top, W = 1, 4, 2, 256, 64, 16, 3, 32
    x = torch.randn((B, N, Hq + 2 * Hkv, d), generator=g, device="cuda").transpose(1, 2)
    q, k, v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:].contiguous()
    wq, wk = [1 + 0.2 * torch.randn(d, generator=g, device="cuda") for _ in range(2)]
    kw = dict(scaling="hope", train_len=128.0)
    rope, (freq, ms) = hb.rope(d, **kw), ref.frequencies(d, **kw)
    pos = torch.arange(N)[None]
    qn, kn = hb.qk_norm_rope(q, k, wq, wk, rope)
    q_lm = torch.randn((B, Hkv, N // S, d), generator=g, device="cuda")
    k_lm, b_lm = hb.landmarks(q_lm, kn, S=S)
    arg = dict(S=S, K_top=K_top, W=W)
    out, _, idx = hb.forward(qn, qn, kn, v, k_lm, b_lm, **arg)
    dout = torch.randn(out.shape, generator=g, device="cuda")
    grads = hb.backward(qn, qn, kn, v, k_lm, b_lm, idx, dout, **arg)
    got = hb.qk_norm_rope_backward(q, k, wq, wk, grads["dq"] + grads["dq_cal"], grads["dK"], rope)
    f = parity.f64
    want = oracle.backward(f(qn), f(qn), f(kn), f(v), f(k_lm), f(b_lm), idx.cpu().numpy(),
                           f(dout), **arg)
    dq = torch.from_numpy(want["dq"] + want["dqc"])
    dk = torch.from_numpy(want["dK"])
    # the attention's gradients arrive within 3e-5 of their plane's largest value (the bound of
    # its own tests); turned back, a pair's errors add to at most sqrt(2) of that
    eq = 3e-5 * math.sqrt(2) * float(abs(want["dq"]).max() + abs(want["dqc"]).max())
    ek = 3e-5 * math.sqrt(2) * float(abs(want["dK"]).max())
    for xx, w, dy, e, n in ((q, wq, dq, eq, "q"), (k, wk, dk, ek, "k")):
        xx, w = xx.double().cpu(), w.double().cpu()
        dx, dw, bx, bw = ref.norm_rope_backward(xx, w, pos, dy, freq, ms, "half")
        # dx = r (h - x r^2 mean(h x)) with |x r| <= sqrt(d) and mean|x r| <= 1
        r = torch.rsqrt(xx.square().mean(-1, keepdim=True) + 1e-6)
        ref.within(got["d" + n], dx, bx + r * e * float(w.abs().max()) * (1 + math.sqrt(d)))
        ref.within(got["dw_" + n], dw, bw + e * (xx * r).abs().sum((0, 1, 2)))
