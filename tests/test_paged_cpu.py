"""Host side of the norms with rotary positions and of the paged cache: hils_rope_init's rules,
argument checks of the C entries (answered before anything touches a device), and the 64-bit
references of the GPU tests against differences and hand-worked cases."""
import ctypes
import math

import pytest
import torch

import ref_paged as ref
from hierarchical_chunk_sparse_scoring_b200 import binding as hb
from hierarchical_chunk_sparse_scoring_b200 import build as hbuild

OK = ctypes.c_void_p(4096)      # never dereferenced: the calls below return before any launch
ODD = ctypes.c_void_p(4100)
R = ctypes.byref


@pytest.fixture(scope="module")
def lib():
    hbuild.build()
    return hb.lib()


@pytest.mark.parametrize("kw", [
    dict(), dict(base=500000.0), dict(scaling="linear", factor=8.0),
    dict(scaling="ntk", factor=4.0), dict(scaling="yarn", factor=16.0, train_len=4096.0),
    dict(scaling="yarn", factor=8.0, train_len=8192.0, beta_fast=4.0, beta_slow=1.0),
    dict(scaling="hope", train_len=1000.0), dict(scaling="hope", train_len=-1.0)],
    ids=lambda k: "-".join(str(v) for v in k.values()) or "plain")
@pytest.mark.parametrize("rot", [0, 16, 64, 128, 256])
def test_rope_init(lib, rot, kw):
    r = hb.rope(rot, layout="interleaved", **kw)
    freq, ms = ref.frequencies(rot, **kw)
    assert r.rot_dim == rot and r.layout == 1 and abs(r.mscale - ms) <= 2 ** -24 * ms
    for m in range(rot // 2):     # pow and a few products in fp64
        assert abs(r.freq[m] - freq[m]) <= 1e-13 * abs(freq[m])
    assert all(f == 0 for f in r.freq[rot // 2:])


def test_rope_own_frequencies(lib):
    r = hb.rope(16, freq=[0.5] * 8, mscale=2.0)
    assert list(r.freq[:8]) == [0.5] * 8 and r.mscale == 2.0
    with pytest.raises(ValueError):
        hb.rope(16, freq=[0.5] * 7)


def test_rope_refusals(lib):
    for kw in (dict(rot_dim=8), dict(rot_dim=272), dict(rot_dim=-16), dict(base=1.0),
               dict(base=math.nan), dict(base=math.inf), dict(scaling="linear", factor=0.5),
               dict(scaling="ntk", factor=math.nan), dict(scaling="yarn", train_len=0.0),
               dict(scaling="yarn", train_len=10.0, beta_fast=1.0, beta_slow=1.0),
               dict(scaling="hope", train_len=math.nan)):
        with pytest.raises(hb.HilsError):
            hb.rope(kw.pop("rot_dim", 64), **kw)
    with pytest.raises(ValueError):
        hb.rope(64, layout="pairs")
    with pytest.raises(ValueError):
        hb.rope(64, scaling="cubic")


def qk(**kw):
    p = hb.QkParams(B=1, N=4, Hq=2, Hkv=1, d=64, dtype=1, grad_dtype=0, norm=1, eps=1e-6)
    for n in ("q", "k", "v", "qo", "ko", "dq", "dk"):
        setattr(p, n + "_str", hb._Strides(0, 256, 64))
    for n, v in kw.items():
        setattr(p, n, hb._Strides(*v) if isinstance(v, tuple) else v)
    return p


QK_BAD = [
    (dict(d=60), 2), (dict(d=264), 2), (dict(d=0), 1), (dict(B=-1), 1), (dict(N=-1), 1),
    (dict(Hq=-1), 1), (dict(Hq=1 << 17), 2), (dict(B=1 << 20, N=1 << 20), 2), (dict(pos0=-1), 1),
    (dict(pos0=1 << 31), 2), (dict(dtype=2), 1), (dict(norm=2), 1), (dict(eps=-1.0), 1),
    (dict(eps=math.nan), 1), (dict(q_str=(0, 257, 64)), 1), (dict(q_str=(0, -64, 64)), 1),
    (dict(ko_str=(0, 0, 32)), 1), (dict(qo_str=(0, 0, 64)), 1), (dict(d=48), 1),
    (dict(q_str=(0, 1 << 62, 64)), 1),
]


@pytest.mark.parametrize("kw,status", QK_BAD, ids=[str(b[0]) for b in QK_BAD])
def test_qk_norm_rope_refuses(lib, kw, status):
    rope = hb.rope(64)
    assert lib.hils_qk_norm_rope(R(qk(**kw)), R(rope), OK, OK, OK, OK, OK, OK, OK, None) == status


def test_qk_norm_rope_pointer_checks(lib):
    rope, p = hb.rope(64), qk()
    f = lib.hils_qk_norm_rope
    assert f(None, R(rope), *[OK] * 7, None) == 1
    assert f(R(p), None, *[OK] * 7, None) == 1
    for i in (0, 1, 5, 6):      # q, k, q_out, k_out: missing, misaligned
        for bad in (None, ODD):
            a = [OK] * 7
            a[i] = bad
            assert f(R(p), R(rope), *a, None) == 1
    assert f(R(p), R(rope), OK, OK, ODD, OK, OK, OK, OK, None) == 1
    assert f(R(p), R(rope), OK, OK, OK, OK, ctypes.c_void_p(4098), OK, OK, None) == 1
    assert f(R(qk(norm=0)), R(rope), OK, OK, OK, None, OK, OK, OK, None) == 1
    for bad in (dict(mscale=math.inf), dict(layout=2), dict(rot_dim=24), dict(rot_dim=-16)):
        r = hb.rope(64)
        for n, v in bad.items():
            setattr(r, n, v)
        assert f(R(p), R(r), *[OK] * 7, None) in (1, 2)
    r = hb.rope(64)
    r.freq[3] = math.nan
    assert f(R(p), R(r), *[OK] * 7, None) == 1
    # nothing to do: no device is touched
    assert f(R(qk(N=0)), R(rope), *[None] * 7, None) == 0
    assert f(R(qk(Hq=0, Hkv=0)), R(rope), *[None] * 7, None) == 0


def test_qk_backward_checks(lib):
    rope, p = hb.rope(64), qk()
    size = lib.hils_qk_backward_workspace_size(R(p))
    assert size > 0 and lib.hils_qk_backward_workspace_size(R(qk(d=60))) == 0
    f = lib.hils_qk_norm_rope_backward
    args = [OK] * 11
    assert f(R(p), R(rope), *args, OK, size - 1, None) == 3
    assert f(R(p), R(rope), *args, None, size, None) == 3
    assert f(R(qk(grad_dtype=1, dtype=0)), R(rope), *args, OK, size, None) == 1
    assert f(R(qk(dq_str=(0, 0, 64))), R(rope), *args, OK, size, None) == 1
    assert f(R(qk(norm=0)), R(rope), *args, OK, size, None) == 1
    assert f(R(qk(N=0)), R(rope), *[None] * 11, None, 0, None) == 0
    for i in (0, 1, 5, 6, 7, 8):
        a = list(args)
        a[i] = ODD
        assert f(R(p), R(rope), *a, OK, size, None) == 1


def cache(**kw):
    c = hb.PagedParams(T=4, B=4, Hq=2, Hkv=1, d=64, n_pages=8, max_pages=4, page_size=16, dtype=1)
    c.c_str = hb._Strides(1024, 1024, 64)
    for n, v in kw.items():
        setattr(c, n, hb._Strides(*v) if isinstance(v, tuple) else v)
    return c


CACHE_BAD = [(dict(T=-1), 1), (dict(B=-1), 1), (dict(n_pages=-1), 1), (dict(max_pages=-1), 1),
             (dict(page_size=0), 1), (dict(window=-1), 1), (dict(n_pages=1 << 28), 2),
             (dict(T=1 << 31), 2), (dict(max_pages=1 << 32), 2)]


@pytest.mark.parametrize("kw,status", CACHE_BAD, ids=[str(b[0]) for b in CACHE_BAD])
def test_paged_calls_refuse(lib, kw, status):
    c = cache(**kw)
    assert lib.hils_paged_workspace_size(R(c)) == 0
    assert lib.hils_paged_plan(R(c), *[OK] * 12, 1 << 30, None) == status
    assert lib.hils_paged_attn(R(c), *[OK] * 9, 1 << 30, None) == status
    assert lib.hils_paged_append(R(qk(N=4)), R(hb.rope(64)), R(c), *[OK] * 11, 1 << 30,
                                 None) == status


def test_paged_plan_checks(lib):
    f = lib.hils_paged_plan
    assert f(R(cache(B=8193)), *[OK] * 12, 256, None) == 2
    assert f(R(cache()), *[OK] * 12, 255, None) == 3
    for i in range(11):
        for bad in (None, ctypes.c_void_p(4098)):
            a = [OK] * 12
            a[i] = bad
            assert f(R(cache()), *a, 256, None) == 1, i
    assert f(R(cache()), *[OK] * 11, None, 256, None) == 3


def test_paged_append_checks(lib):
    f, rope = lib.hils_paged_append, hb.rope(64)
    for kw in (dict(T=5), dict(Hq=3), dict(Hkv=2), dict(d=128), dict(dtype=0)):
        assert f(R(qk()), R(rope), R(cache(**kw)), *[OK] * 11, 256, None) == 1
    assert f(R(qk(B=2, N=2)), R(rope), R(cache()), *[OK] * 11, 256, None) == 1
    assert f(R(qk()), R(rope), R(cache(c_str=(1024, 1024, 32))), *[OK] * 11, 256, None) == 1
    assert f(R(qk()), R(rope), R(cache(c_str=(1024, 1024, 65))), *[OK] * 11, 256, None) == 1
    assert f(R(qk()), R(rope), R(cache()), *[OK] * 11, 255, None) == 3
    for i in (0, 1, 2, 5, 6, 7, 8, 9):
        a = [OK] * 11
        a[i] = None
        assert f(R(qk()), R(rope), R(cache()), *a, 256, None) == 1, i


def test_paged_attn_checks(lib):
    f = lib.hils_paged_attn
    big = 1 << 30
    size = lib.hils_paged_workspace_size(R(cache()))
    assert size > 256 and lib.hils_paged_workspace_size(R(cache(d=96))) == 256
    for kw, status in ((dict(Hq=3, Hkv=2), 1), (dict(Hq=0), 1), (dict(d=96), 2),
                       (dict(Hq=17, Hkv=1), 2), (dict(dtype=3), 1), (dict(scale=math.nan), 1),
                       (dict(c_str=(1024, 1024, 4)), 1)):
        assert f(R(cache(**kw)), *[OK] * 9, big, None) == status, kw
    assert f(R(cache()), *[OK] * 9, size - 1, None) == 3
    a = [OK] * 9
    a[4] = None     # rows are sequences: no more of them than table rows
    assert f(R(cache(T=5)), *a, big, None) == 1
    for i in (0, 1, 2, 3, 5, 6):
        a = [OK] * 9
        a[i] = None
        assert f(R(cache()), *a, big, None) == 1, i
    assert f(R(cache(T=0)), *[None] * 8, OK, big, None) == 0


# ------------------------------------------------------------------- the references themselves

@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_reference_gradient_matches_differences(layout):
    g = torch.Generator().manual_seed(1)
    x, dy = [torch.randn((2, 3, 4, 40), generator=g, dtype=torch.float64) for _ in range(2)]
    w = torch.randn(40, generator=g, dtype=torch.float64)
    pos = torch.randint(0, 1000, (2, 4), generator=g)
    freq, ms = ref.frequencies(32, "yarn", factor=4.0, train_len=512.0)
    dx, dw, _, _ = ref.norm_rope_backward(x, w, pos, dy, freq, ms, layout)
    f = lambda x, w: (ref.norm_rope(x, w, pos, freq, ms, layout)[0] * dy).sum()
    h = 1e-6
    for _ in range(4):
        ex, ew = torch.randn(x.shape, generator=g).double(), torch.randn(40, generator=g).double()
        diff = (f(x + h * ex, w + h * ew) - f(x - h * ex, w - h * ew)) / (2 * h)
        assert abs(float(diff - (dx * ex).sum() - (dw * ew).sum())) <= 1e-6 * float(dy.abs().sum())


def test_reference_rotation_by_hand():
    x = torch.tensor([[[[3.0, 4.0, 5.0, 7.0]]]], dtype=torch.float64)
    quarter = [math.pi / 2, math.pi / 2]
    p = torch.tensor([[1]])
    y, _ = ref.norm_rope(x, None, p, quarter, 1.0, "half", norm=False)
    assert torch.allclose(y.flatten(), torch.tensor([-5.0, -7.0, 3.0, 4.0]).double())
    y, _ = ref.norm_rope(x, None, p, quarter, 1.0, "interleaved", norm=False)
    assert torch.allclose(y.flatten(), torch.tensor([-4.0, 3.0, -7.0, 5.0]).double())
    w = torch.tensor([1.0, 2.0, 1.0, 1.0]).double()
    y, _ = ref.norm_rope(x[..., :2], w[:2], p, [], 1.0, "half", eps=0.0)
    assert torch.allclose(y.flatten(), torch.tensor([3.0, 8.0]).double() / math.sqrt(12.5))


def test_reference_plan_by_hand():
    got, bad = ref.plan([3, 8, 0], [2, 1, 0], [[4, -1], [1, -1], [-1, -1]], [0, 2, 3], 3, 4, 5, 8)
    # 3 tokens + 2 need a second page of 4; 8 tokens fill their two pages and outgrow the row
    assert bad and got["kv_len"] == [5, 8, 0] and got["n_free"] == [2]
    assert got["slot"] == [19, 12, -1, -1, -1] and got["pos"][:2] == [3, 4]
    assert got["table"][0] == [4, 3] and got["cu"] == [0, 2, 2, 2]


def test_reference_attention_by_hand():
    q = torch.tensor([[1.0, 0.0]]).double()
    K = torch.tensor([[[math.log(2.0), 5.0]], [[0.0, 1.0]], [[math.nan, 0.0]]]).double()
    V = torch.tensor([[[3.0, 0.0]], [[0.0, 6.0]], [[1.0, 1.0]]]).double()
    out, lse, _, _ = ref.attention(q, K, V, 0, 2, 1.0, torch.float32)
    assert torch.allclose(out[0], torch.tensor([2.0, 2.0]).double())
    # ln 2 is given in fp32, within 2^-25; its weight is 2/3
    assert abs(float(lse) - math.log(3.0)) <= 2 / 3 * 2 ** -25 + 1e-15


def test_binding_has_no_cpu_path(lib):
    q = torch.zeros((1, 2, 4, 64))
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError):
        hb.qk_norm_rope(q, None, None, None, hb.rope(64))
    with pytest.raises(ValueError):
        hb.paged_plan(i, i, torch.zeros((4, 2), dtype=torch.int32), i, i[:1], page_size=4, T_cap=4)
    with pytest.raises(ValueError):
        hb.paged_attn(q[0].transpose(0, 1).contiguous(), q, q, i.view(4, 1), i)
