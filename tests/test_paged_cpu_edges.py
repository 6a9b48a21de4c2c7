"""Host side: arrays of a call that lie over one another.  A plan of more than one block reads the
lengths in every block while the first one writes the new ones, and an operator in place reads each
element in the lane that writes it, so other overlaps would race on the device: they are refused
before any launch."""
import ctypes

import pytest

from hierarchical_chunk_sparse_scoring_b200 import binding as hb
from hierarchical_chunk_sparse_scoring_b200 import build as hbuild
from test_paged_cpu import R, cache, qk

BAD = 1


@pytest.fixture(scope="module")
def lib():
    hbuild.build()
    return hb.lib()


def at(n):
    return ctypes.c_void_p(n << 16)     # (never dereferenced: every call below is refused)


# kv_len, new_len, block_table, free_pages, n_free, kv_len_out, n_free_out, cu, slot, pos, seq
PLAN = [at(i + 1) for i in range(11)]


@pytest.mark.parametrize("i,j,shift", [
    (5, 1, 0), (5, 3, 0), (5, 4, 0), (6, 0, 0), (6, 1, 4), (6, 3, 28), (7, 0, 0), (8, 1, 0), (9, 0, 4),
    (10, 3, 0), (2, 1, 0), (2, 0, 12), (5, 0, 4), (0, 5, 4), (8, 9, 0), (9, 10, 12), (10, 7, 16),
    (8, 2, 60), (5, 6, 0), (7, 5, 8), (3, 2, 0)])
def test_plan_refuses_arrays_over_one_another(lib, i, j, shift):
    """Array i begins `shift` bytes into array j."""
    a = list(PLAN)
    a[i] = ctypes.c_void_p(a[j].value + shift)
    assert lib.hils_paged_plan(R(cache()), *a, at(12), 256, None) == BAD


def test_norm_refuses_tensors_over_one_another(lib):
    rope, f = hb.rope(64), lib.hils_qk_norm_rope
    q, k, qo, ko, w = [at(i) for i in range(1, 6)]

    def go(q, k, qo, ko, **kw):
        return f(R(qk(**kw)), R(rope), q, k, w, w, w, qo, ko, None)
    assert go(q, k, q, ko, qo_str=(0, 512, 64)) == BAD      # in place, other strides
    assert go(q, k, qo, k, ko_str=(0, 256, 128)) == BAD
    assert go(q, k, k, ko) == BAD
    assert go(q, k, qo, q) == BAD
    assert go(q, k, qo, qo) == BAD


def test_norm_backward_refuses_tensors_over_one_another(lib):
    rope, f = hb.rope(64), lib.hils_qk_norm_rope_backward
    size = lib.hils_qk_backward_workspace_size(R(qk()))
    names = ("q", "k", "w_q", "w_k", "pos", "dq_out", "dk_out", "dq", "dk", "dw_q", "dw_k")

    def go(p, **same):
        a = {n: at(i + 1) for i, n in enumerate(names)}
        for n, m in same.items():
            a[n] = a[m]
        return f(R(p), R(rope), *[a[n] for n in names], at(20), size, None)
    assert go(qk(dq_str=(0, 512, 64)), dq="dq_out") == BAD
    assert go(qk(dk_str=(0, 256, 128)), dk="dk_out") == BAD
    assert go(qk(dq_str=(0, 512, 64), grad_dtype=1), dq="q") == BAD
    assert go(qk(), dq="q") == BAD                          # fp32 over bf16
    for n, m in (("dq", "dk"), ("dq", "dk_out"), ("dk", "dq_out"), ("dq", "k"), ("dk", "q"),
                 ("dw_q", "dw_k")):
        assert go(qk(grad_dtype=1), **{n: m}) == BAD, (n, m)


def test_append_refuses_tensors_over_one_another(lib):
    rope, f = hb.rope(64), lib.hils_paged_append
    names = ("q", "k", "v", "w_q", "w_k", "pos", "slot", "q_out", "K", "V")

    def go(p, **same):
        a = {n: at(i + 1) for i, n in enumerate(names)}
        for n, m in same.items():
            a[n] = a[m]
        return f(R(p), R(rope), R(cache()), *[a[n] for n in names], at(20), 256, None)
    assert go(qk(qo_str=(0, 512, 64)), q_out="q") == BAD
    for n, m in (("q_out", "k"), ("q_out", "v"), ("K", "V")):
        assert go(qk(), **{n: m}) == BAD, (n, m)
