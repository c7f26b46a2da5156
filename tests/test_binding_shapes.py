"""What the library cannot see of the tensors it gets as pointers: the binding of the
reading back and of the rotating append refuses lengths that would be read or written
past their end.  The plans are host plans, so nothing reaches a GPU."""
import pytest

from asymmetric_kv_paged_gb300 import binding as B

torch = pytest.importorskip("torch")


def host_plan(qo=(0, 2, 3), seq=(20, 9), **kw):
    prob, keep = B.make_problem(batch=len(seq), num_q_heads=8, num_kv_heads=1, page_size=16, num_pages=9,
                                page_table_stride=4, kv_dtype=B.ATTN_KV_FP4_E2M1, window=0, has_sinks=False,
                                qo_indptr=list(qo), seq_lens=list(seq))
    return B.attn_plan_host(prob, 152, keep if kw.get("keep", True) else None)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


T = torch.zeros(16, dtype=torch.int32)


@pytest.mark.parametrize("k,v", [(5, 4), (4, 5), (5, 0)])
def test_read_needs_as_many_value_rows_as_key_rows(k, v):
    with pytest.raises(ValueError):
        B.attn_read_kv(host_plan(), T, T, T, T, T, bf(k, 1, 192), bf(v, 1, 128))


def test_read_with_equal_rows_reaches_the_library():
    with pytest.raises(B.AttnError) as e:                 # which refuses the host plan
        B.attn_read_kv(host_plan(), T, T, T, T, T, bf(4, 1, 192), bf(4, 1, 128))
    assert e.value.status == B.ATTN_ERR_INVALID_ARG


def append(plan, positions):
    rope = B.make_rope(torch.zeros(30, 64), 64, positions=positions)
    B.attn_append_kv_rope(plan, rope, None, bf(3, 1, 192), bf(3, 1, 128), None, T, T, T, T, T)


@pytest.mark.parametrize("n", [0, 1, 2])
def test_positions_shorter_than_the_plans_tokens_are_refused(n):
    with pytest.raises(ValueError):
        append(host_plan(), torch.zeros(n, dtype=torch.int32))


@pytest.mark.parametrize("n", [3, 4, None])
def test_positions_of_every_token_reach_the_library(n):
    with pytest.raises(B.AttnError) as e:
        append(host_plan(), None if n is None else torch.zeros(n, dtype=torch.int32))
    assert e.value.status == B.ATTN_ERR_INVALID_ARG


def test_plans_know_their_tokens():
    assert host_plan().total_q == 3
    assert host_plan((0, 0, 0)).total_q == 0
    assert host_plan((0,), ()).total_q == 0
    prob, keep = B.make_problem(batch=1, num_q_heads=8, num_kv_heads=1, page_size=16, num_pages=9,
                                page_table_stride=4, kv_dtype=B.ATTN_KV_BF16, window=0, has_sinks=False,
                                qo_indptr=[0, 7], seq_lens=[20])
    assert B.attn_plan_replayable_host(prob, 152, keep).total_q == 7
