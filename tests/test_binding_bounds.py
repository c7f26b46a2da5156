"""Bounds arrays and what is read of them: the binding refuses arrays of another block size, type or
order than the call's, which would be read or written past their end.  The plans are host plans
that the binding takes for device plans, so nothing reaches a GPU: what it lets through the library
refuses."""
import pytest

from asymmetric_kv_paged_gb300 import binding as B

torch = pytest.importorskip("torch")

T = torch.zeros(16, dtype=torch.int32)
U8 = torch.uint8


def plan(page_size=128, head_dim=192, replayable=False):
    prob, keep = B.make_problem(batch=2, num_q_heads=16, num_kv_heads=2, page_size=page_size, num_pages=5,
                                page_table_stride=8, kv_dtype=B.ATTN_KV_BF16, window=0, has_sinks=False,
                                qo_indptr=[0, 1, 3], seq_lens=[100, 120], head_dim_qk=head_dim)
    p = (B.attn_plan_replayable_host if replayable else B.attn_plan_host)(prob, 152, keep)
    p.device = 0
    return p


def calls(p, block, bounds):
    idx = torch.zeros(3, 2, 4, dtype=torch.int32)
    out = torch.zeros(1, 2, 2, p.head_dim_qk, dtype=torch.bfloat16)
    return (lambda: B.attn_update_bounds(p, block, T, bounds, T, T, T, 3, stream=0),
            lambda: B.attn_read_bounds(p, block, bounds, T, T, T, out, stream=0),
            lambda: B.attn_select_blocks(p, B.make_sparse(block, 4), T, bounds, T, T, T, idx, stream=0))


def refused(call):
    with pytest.raises(ValueError):
        call()


def reaches_the_library(call):
    with pytest.raises(B.AttnError) as e:
        call()
    assert e.value.status == B.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("head_dim,row", [(192, 400), (128, 272)])
@pytest.mark.parametrize("replayable", [False, True])
def test_arrays_of_another_block_size_type_or_order(head_dim, row, replayable):
    p = plan(head_dim=head_dim, replayable=replayable)
    for block in (16, 32, 64, 128):
        good = torch.zeros(5, 128 // block, 2, row, dtype=U8)
        for call in calls(p, block, good):
            reaches_the_library(call)
        for bad in (torch.zeros(5, 128 // block, 2, row - 1, dtype=U8), torch.zeros(4, 128 // block, 2, row, dtype=U8),
                    torch.zeros(5, 128 // block, 1, row, dtype=U8), good.view(torch.int8), good.float(),
                    torch.zeros(128 // block, 5, row, 2, dtype=U8).transpose(2, 3),
                    torch.zeros(10, 128 // block, 2, row, dtype=U8)[::2]):
            for call in calls(p, block, bad):
                refused(call)
    for call in calls(p, 16, torch.zeros(5, 2, 2, row, dtype=U8)):          # of blocks of 64
        refused(call)


def test_longer_arrays_and_what_the_library_refuses_itself():
    p = plan()
    for call in calls(p, 64, torch.zeros(9, 2, 2, 400, dtype=U8)):           # a pool of more pages
        reaches_the_library(call)
    for call in (*calls(p, 64, None), *calls(p, 24, T), *calls(plan(page_size=48), 32, T)):
        reaches_the_library(call)
    p.device = -1
    for call in calls(p, 64, T):
        reaches_the_library(call)


def test_bounds_read_back_into_another_shape():
    p, bounds = plan(), torch.zeros(5, 2, 2, 400, dtype=U8)
    for out in (None, torch.zeros(3, 2, 192, dtype=torch.bfloat16), torch.zeros(3, 2, 2, 128, dtype=torch.bfloat16),
                torch.zeros(3, 1, 2, 192, dtype=torch.bfloat16), torch.zeros(3, 2, 2, 192)):
        refused(lambda: B.attn_read_bounds(p, 64, bounds, T, T, T, out, stream=0))
    reaches_the_library(lambda: B.attn_read_bounds(p, 64, bounds, T, T, T, torch.zeros(3, 2, 2, 192, dtype=torch.bfloat16),
                                                   stream=0))
