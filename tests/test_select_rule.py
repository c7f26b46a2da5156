"""Which kernel attn_select_blocks launches, from the plan alone (no GPU)."""
import numpy as np
import pytest

from asymmetric_kv_paged_gb300 import binding as B


def ctas(seq, n, hq=16, hkv=4, block=16, take=9, first=1, dqk=192, num_sms=152, window=0, replayable=False):
    prob, keep = B.make_problem(batch=len(seq), num_q_heads=hq, num_kv_heads=hkv, page_size=128, num_pages=10000,
                                page_table_stride=(max(seq) + 127) // 128, kv_dtype=B.ATTN_KV_BF16, window=window,
                                has_sinks=False, qo_indptr=np.concatenate([[0], np.cumsum(n)]), seq_lens=seq,
                                head_dim_qk=dqk)
    plan = (B.attn_plan_replayable_host if replayable else B.attn_plan_host)(prob, num_sms, keep)
    return B.attn_plan_select_ctas(plan, B.make_sparse(block, take, first, 1))


@pytest.mark.parametrize("replayable", [False, True])
@pytest.mark.parametrize("hq,hkv,dqk", [(8, 4, 128), (64, 4, 192), (160, 4, 192)])
def test_clusters_by_the_longest_request(hq, hkv, dqk, replayable):
    """256 scored blocks a CTA, eight CTAs at most; the first blocks are not scored."""
    for blocks, want in ((257, 1), (258, 2), (513, 2), (514, 3), (1793, 7), (1794, 8), (2048, 8), (2049, 8), (2050, 0),
                         (2063, 0), (8000, 0)):
        assert ctas([16 * blocks, 300], [200, 200], hq, hkv, dqk=dqk, replayable=replayable) == want, blocks
    assert ctas([16 * 2050], [200], hq, hkv, first=2, dqk=dqk) == 8


def test_tokens_a_request_and_in_all():
    assert ctas([2000] * 200, [1] * 200) == 0                      # fewer than two a request
    assert ctas([2000] * 200, [2] * 200) == 1
    assert ctas([2000] * 200, [3, 1] * 100) == 1
    assert ctas([2000, 2000], [0, 77]) == 1                        # 308 tokens x KV heads, 304 are two an SM
    assert ctas([2000], [76]) == 0
    assert ctas([2000], [76], num_sms=100) == 1
    assert ctas([2000], [0]) == 0
    assert ctas([4000], [400], 128, 1) == 1 and ctas([4000], [400], 129, 1) == 0      # rows of a token tile


def test_refusals():
    for kw, status in ((dict(block=48), B.ATTN_ERR_UNSUPPORTED), (dict(take=257), B.ATTN_ERR_INVALID_ARG),
                       (dict(window=100), B.ATTN_ERR_INVALID_ARG)):
        with pytest.raises(B.AttnError) as e:
            ctas([2000], [200], **kw)
        assert e.value.status == status
    for hq, hkv, blocks in ((16, 4, 49153), (128, 1, 49152)):
        with pytest.raises(B.AttnError) as e:
            ctas([16 * blocks], [200], hq, hkv, dqk=128)
        assert e.value.status == B.ATTN_ERR_UNSUPPORTED
