"""Attention over selected blocks, what needs no GPU: record sizes, what the binding refuses,
the axes helper, and pins of the tests' plain forms."""
import ctypes

import numpy as np
import pytest

import sparse_plain as P_
from asymmetric_kv_paged_gb300 import binding as B
from asymmetric_kv_paged_gb300 import workloads as W

torch = pytest.importorskip("torch")

T = torch.zeros(16, dtype=torch.int32)


def host_plan(page_size=64, window=0):
    prob, keep = B.make_problem(batch=2, num_q_heads=16, num_kv_heads=2, page_size=page_size, num_pages=20,
                                page_table_stride=8, kv_dtype=B.ATTN_KV_BF16, window=window, has_sinks=False,
                                qo_indptr=[0, 1, 3], seq_lens=[100, 120])
    return B.attn_plan_host(prob, 152, keep)


def test_record_sizes():
    assert B.attn_bounds_row_bytes(192) == 400 and B.attn_bounds_row_bytes(128) == 272
    for d in (0, 64, 256):
        with pytest.raises(B.AttnError) as e:
            B.attn_bounds_row_bytes(d)
        assert e.value.status == B.ATTN_ERR_UNSUPPORTED
    assert B.load().attn_bounds_row_bytes(192, ctypes.POINTER(ctypes.c_int32)()) == B.ATTN_ERR_INVALID_ARG


def test_host_plans_are_refused():
    p, s = host_plan(), B.make_sparse(64, 4)
    idx = torch.zeros(3, 2, 4, dtype=torch.int32)
    out = torch.zeros(1, 2, 2, 192, dtype=torch.bfloat16)
    m = B.make_mrope(torch.zeros(30, 64), 64, [0] * 32)
    for call in (lambda: B.attn_update_bounds(p, 64, T, T, T, T, T, 3),
                 lambda: B.attn_read_bounds(p, 64, T, T, T, T, out),
                 lambda: B.attn_select_blocks(p, s, T, T, T, T, T, idx),
                 lambda: B.attn_run_sparse(p, s, T, T, T, T, T, T, idx, None, 1.0, 1.0, 1.0, out),
                 lambda: B.attn_append_kv_mrope(p, m, None, T, T, None, T, T, T, T, T)):
        with pytest.raises(B.AttnError) as e:
            call()
        assert e.value.status == B.ATTN_ERR_INVALID_ARG


def test_list_arrays_of_another_size_are_refused():
    p, s = host_plan(), B.make_sparse(64, 4)
    for shape in ((3, 2, 3), (2, 2, 4), (3, 1, 4), (4, 2, 4)):
        idx = torch.zeros(shape, dtype=torch.int32)
        with pytest.raises(ValueError):
            B.attn_select_blocks(p, s, T, T, T, T, T, idx)
        with pytest.raises(ValueError):
            B.attn_run_sparse(p, s, T, T, T, T, T, T, idx, None, 1.0, 1.0, 1.0, T)


def test_list_arrays_of_another_type_or_order_are_refused():
    p, s = host_plan(), B.make_sparse(64, 4)
    for idx in (torch.zeros(3, 2, 4, dtype=torch.int64), torch.zeros(3, 2, 4),
                torch.zeros(2, 3, 4, dtype=torch.int32).transpose(0, 1)):
        with pytest.raises(ValueError):
            B.attn_select_blocks(p, s, T, T, T, T, T, idx)
        with pytest.raises(ValueError):
            B.attn_run_sparse(p, s, T, T, T, T, T, T, idx, None, 1.0, 1.0, 1.0, T)


def test_axes():
    assert B.mrope_axes([2, 3, 1]) == [0, 0, 1, 1, 1, 2]
    assert B.mrope_axes([2, 3, 1], in_turn=True) == [0, 1, 2, 0, 1, 1]
    tab = torch.zeros(30, 64)
    for axes in ([0] * 31, [0] * 33, [-1] * 32, []):
        with pytest.raises(ValueError):
            B.make_mrope(tab, 64, axes)
    axes = B.mrope_axes([8, 12, 12])
    for pos in (torch.zeros(2, 5, dtype=torch.int32), torch.zeros(3, 5), torch.zeros(15, dtype=torch.int32),
                torch.zeros(5, 3, dtype=torch.int32).T):
        with pytest.raises(ValueError):
            B.make_mrope(tab, 64, axes, positions=pos)
    with pytest.raises(ValueError):
        B.make_mrope(tab, 64, axes, position_delta=torch.zeros(2))
    p = host_plan()
    for kw in (dict(positions=torch.zeros(3, 2, dtype=torch.int32)), dict(positions=torch.zeros(3, 4, dtype=torch.int32)),
               dict(position_delta=torch.zeros(1, dtype=torch.int32))):
        with pytest.raises(ValueError):
            B.attn_append_kv_mrope(p, B.make_mrope(tab, 64, axes, **kw), None, T, T, None, T, T, T, T, T)
    assert B.make_mrope(tab, 64, axes, positions=torch.zeros(4, 3, dtype=torch.int32)).num_axes == 4


def test_plain_exponent_and_record():
    assert [P_.exponent(a) for a in (0.0, 1.0, 127.0, 127.5, 128.0, 1.984375, 1.9921875)] == [0, -6, 0, 1, 1, -6, -5]
    rec = P_.record(np.array([[1.0, -2.0, 0.3], [0.5, -1.0, 0.1]]), 16).view(np.int8)
    # max |k| = 2 = 64 / 32: unit 2^-5
    assert rec[:7].tolist() == [32, -32, 10, 16, -64, 3, -5] and not rec[7:].any()


def test_plain_scores_bound_the_products():
    rng = np.random.default_rng(1)
    q, k = rng.standard_normal((3, 128)), rng.standard_normal((64, 128))
    rec = P_.record(k, 272)[None]
    qi = np.stack([np.rint(x / 2.0 ** P_.exponent(np.abs(x).max())) for x in q])
    unit = [2.0 ** P_.exponent(np.abs(x).max()) for x in q]
    best = max((qi[h] @ k.T).max() * unit[h] / max(unit) for h in range(3))
    assert P_.scores(q, rec, 128)[0] >= best


def test_plain_choice():
    s = np.array([0.0, 5, 9, 9, 1, 9, 0, 0])
    assert P_.choose(s, 7, 4, 1, 1).tolist() == [0, 2, 3, 7]
    assert P_.choose(s, 7, 5, 1, 1).tolist() == [0, 2, 3, 5, 7]
    assert P_.choose(s, 2, 5, 1, 1).tolist() == [0, 1, 2, -1, -1]
    assert P_.choose(s, 7, 3, 0, 3).tolist() == [5, 6, 7]


def test_plain_attention_with_all_blocks_is_the_oracles():
    from oracle import oracle
    w = W.make_workload(5, [70, 33], [3, 1], hq=4, hkv=2, page_size=16, kv_dtype="bf16", sinks=True)
    lists = np.broadcast_to(np.arange(5, dtype=np.int32), (4, 2, 5))
    ref, ref_lse = oracle.attn_paged(w.host_arrays())
    out, lse = P_.attend(w, w.q, 16, lists, w.sinks)[:2]
    # the oracle takes fp32 scalars (softmax scale, sinks) and returns fp64 sums in another order
    assert np.allclose(out, ref, rtol=0, atol=1e-6) and np.allclose(lse, ref_lse, rtol=0, atol=1e-6)
