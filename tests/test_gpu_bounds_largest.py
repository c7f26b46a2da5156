"""Bounds of the largest bf16 values: records, what they read back as, lists chosen by them."""
import numpy as np
import pytest

import sparse_plain as P_
from asymmetric_kv_paged_gb300 import workloads as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_bounds import device, indptr, setup, update  # noqa: E402


def test_bounds_past_the_largest_bf16_read_back_as_infinities():
    """max |k| up to 127 * 2^121 has the unit 2^121 and reads back exactly; above it the unit is
    2^122, and a code of +-64 stands for +-2^128, which bf16 does not hold."""
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw, row = setup("bf16", [64 * 4], [1], 64)
    k = w.k_cache.reshape(-1, 2, 192).copy()
    s = [int(P_.slots(w, 0, 64 * c)) for c in range(4)]
    k[s[0] + 1, 0, 3] = 0x7F7E                                   # 127 * 2^121
    k[s[1] + 1, 0, 3] = 0x7F7F                                   # 127.5 * 2^121: 64 units of 2^122, rounded up
    k[s[2] + 9, 0, 7] = 0xFF7F
    k[s[2] + 9, 0, 8] = 0x7F7C                                   # 126 * 2^121 beside it: 63 units, exact
    k[s[3]:s[3] + 64, 0] = 0xFF7F
    dw.k_cache.copy_(torch.from_numpy(k.view(np.int16)).view(torch.bfloat16).cuda().view(dw.k_cache.shape))
    bounds = torch.zeros(w.num_pages, 1, 2, row, dtype=torch.uint8, device="cuda")
    ind = indptr([64 * 4])
    update(dw, 64, bounds, ind)
    kc = k.reshape(w.k_cache.shape)
    ref = P_.update_bounds(w, np.zeros(bounds.shape, np.uint8), 64, kc, w.seq_lens, ind)
    assert np.array_equal(bounds.cpu().numpy(), ref)
    out = torch.empty(4, 2, 2, 192, dtype=torch.bfloat16, device="cuda")
    B.attn_read_bounds(dw.plan, 64, bounds, dw.page_table, dw.seq_lens, device(indptr([4])), out)
    assert B.attn_get_device_error(dw.plan) == 0
    got = out.double().cpu().numpy()
    r = ref.reshape(-1, 2, row).view(np.int8).astype(np.float64)[np.array(s) // 64]
    with np.errstate(over="ignore"):
        want = r[..., :384].reshape(4, 2, 2, 192) * 2.0 ** r[..., 384][..., None, None]
    want[np.abs(want) >= 2.0 ** 128] = np.inf * np.sign(want[np.abs(want) >= 2.0 ** 128])
    assert np.array_equal(got, want)
    assert got[0, 0, 0, 3] == 127 * 2.0 ** 121 and got[1, 0, 0, 3] == np.inf
    assert got[2, 0, 1, 7] == -np.inf and got[2, 0, 0, 8] == 126 * 2.0 ** 121
    assert (got[3, 0, 1] == -np.inf).all() and (got[3, 0, 0] == -63 * 2.0 ** 122).all()
    assert np.isfinite(got[:, 1]).all()


@pytest.mark.parametrize("n", [1, 200])
def test_scores_past_fp32_are_infinities(n):
    """Units of up to 2^122: scores beyond fp32's range are equal, the lowest blocks first, and
    come before all finite ones (below the range behind them)."""
    from test_gpu_select import random_bounds, run, setup as select_setup
    from test_gpu_select_scales import scores
    w, dw = select_setup([3000], [n], 16, 2, 64)
    rng = np.random.default_rng(6)
    bounds = random_bounds(rng, w, 64).view(np.int8)
    bounds[..., 384] = rng.integers(105, 123, bounds.shape[:-1])
    got = run(w, dw, w.q, bounds.view(np.uint8), 64, 14, 1, 1)
    flat = bounds.view(np.uint8).reshape(-1, 2, bounds.shape[-1])
    at = P_.slots(w, 0, np.arange(47) * 64) // 64
    qv = W.bf16_values(w.q).astype(np.float64)
    many = 0
    for tok in range(n):
        own = (3000 - n + tok) // 64
        for g in range(2):
            with np.errstate(over="ignore"):
                s = scores(qv[tok, 8 * g:8 * g + 8], flat[at[:own + 1], g], 192)
            assert np.array_equal(got[tok, g], P_.choose(s, own, 14, 1, 1)), (tok, g)
            many += np.isinf(s[1:own]).sum() > 3 and np.isfinite(s[1:own]).sum() > 3
    assert many == 2 * n
