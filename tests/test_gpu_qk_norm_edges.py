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
