"""attn_select_blocks for chunks whose blocks seven or eight CTAs share out, the most there are: the
lists equal the definition's, for token tiles of 32, 8 and 2 tokens and beside short requests whose
blocks some of the CTAs have nothing of."""
import numpy as np
import pytest

import sparse_plain as P_

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_select import random_bounds, run, setup  # noqa: E402


@pytest.mark.parametrize("seq,n,hq,hkv,P,dqk,block,take,ctas", [
    ([32768, 700, 20000], [96, 40, 33], 8, 4, 128, 128, 16, 9, 8),         # a token has 4 rows
    ([900, 28000], [20, 110], 48, 3, 64, 192, 16, 40, 7),                  # 16
    ([32768], [310], 40, 1, 32, 128, 16, 200, 8),                          # 64: two tokens a tile, six CTAs without a list
    ([65000, 65000], [80, 75], 16, 2, 64, 192, 32, 3, 8),
    ([33000], [96], 8, 4, 128, 128, 16, 9, 0),                             # one CTA more than eight: token by token
])
def test_lists_over_the_largest_clusters(seq, n, hq, hkv, P, dqk, block, take, ctas):
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup(seq, n, hq, hkv, P, dqk)
    assert B.attn_plan_select_ctas(dw.plan, B.make_sparse(block, take, 1, 2)) == ctas
    bounds = random_bounds(np.random.default_rng(3), w, block)
    got = run(w, dw, w.q, bounds, block, take, 1, 2)
    assert B.attn_get_device_error(dw.plan) == 0
    assert np.array_equal(got, P_.select(w, w.q, bounds, block, take, 1, 2))


def test_ties_over_a_cluster_of_eight():
    """Every block alike: the lowest ones, whichever CTA has them; and two values only."""
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup([32768], [160], 16, 2, 64, 128)
    assert B.attn_plan_select_ctas(dw.plan, B.make_sparse(16, 12, 1, 2)) == 8
    bounds = random_bounds(np.random.default_rng(1), w, 16, spread=2)
    bounds[...] = bounds[:1, :1]
    got = run(w, dw, w.q, bounds, 16, 12, 1, 2)
    assert (got[..., :10] == np.arange(10)).all()
    assert np.array_equal(got, P_.select(w, w.q, bounds, 16, 12, 1, 2))
    two = bounds.view(np.int8).copy()
    two[::7, ..., 256] += 1
    assert np.array_equal(run(w, dw, w.q, two.view(np.uint8), 16, 12, 1, 2),
                          P_.select(w, w.q, two.view(np.uint8), 16, 12, 1, 2))
