"""Rows whose scores are all zero, or whose score scale is below fp32's range, on
8- and 4-bit caches: the mask's -inf stays -inf, and the row is the mean of what it
sees (with the sink's share), on every kernel that a row count picks.

Tolerance per output element, with A the mean of |v| over the visible keys: the
weights are equal and powers of two, so they are exact in 16 bits; the sums' fp32
roundings are below 2^-12 A for the lengths here, the result is rounded to bf16
(2^-8 |out|).  The other rows of a batch have scores up to ~5 and weights of 16
bits (bf16 at worst: 2^-8 A).
"""
import numpy as np
import pytest

from asymmetric_kv_paged_gb300 import workloads as W
from oracle import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -8

# name, seq_lens, n, hq, page size: row blocks of 8 to 256 rows, whole and split
SHAPES = [
    ("rows8", [70, 33], [1, 1], 16, 16),
    ("rows8_long", [9001, 40], [1, 1], 16, 16),
    ("rows16_p1", [90, 700], [2, 2], 16, 1),
    ("rows32_few_tiles", [300, 90], [4, 4], 16, 16),
    ("rows32_long", [16001, 90], [4, 4], 16, 16),
    ("rows64", [330, 72], [8, 8], 16, 128),
    ("rows64_long_p3", [9000], [8], 16, 3),
    ("rows128", [333, 90], [15, 2], 16, 16),
    ("rows256", [300, 90], [200, 60], 16, 16),
    ("rows256_long", [5000], [200], 16, 1),
]


def check(w, out, lse):
    ref, ref_lse = oracle.attn_paged(w.host_arrays())
    mag = w.host_arrays()
    mag["v_cache"] = mag["v_cache"] & (0x7F if w.kv_dtype == "fp8" else 0x7FFF)
    a, _ = oracle.attn_paged(mag)
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got)), f"{np.count_nonzero(~np.isfinite(got).all(-1))} rows are not finite"
    assert np.all(np.abs(got - ref) <= U * (1.1 * a + np.abs(ref)) + 1e-9)
    assert np.abs(lse.cpu().numpy() - ref_lse).max() <= 3e-4


def run(w, **kw):
    from asymmetric_kv_paged_gb300 import binding as B
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    dw = DeviceWorkload(w, **kw)
    dw.out.fill_(float("nan"))
    dw.run()
    torch.cuda.synchronize()
    assert B.attn_get_device_error(dw.plan) == 0
    check(w, dw.out, dw.lse)
    return dw


@pytest.mark.parametrize("kv", ["fp4", "fp8"])
@pytest.mark.parametrize("shape", SHAPES, ids=[s[0] for s in SHAPES])
@pytest.mark.parametrize("sinks", [False, True])
def test_zero_query_rows_among_large_ones(shape, kv, sinks):
    """Queries of 1e18 with a scale of 7e-20 leave a zero row (a padded token, a
    head that is off) and one of subnormals no score scale above fp32's range."""
    name, seq, n, hq, P = shape
    w = W.make_workload(21, seq, n, hq=hq, hkv=2, page_size=P, kv_dtype=kv, sinks=sinks, name=name, q_std=1e18,
                        softmax_scale=float(np.float32(0.07 / 1e18)))
    w.q[0] = 0                                     # a whole token
    w.q[:, 3] = 0x8000                             # a head of -0
    w.q[-1, 5:7] = 0x0001                          # subnormals, the smallest
    run(w)


@pytest.mark.parametrize("kv", ["fp4", "fp8"])
@pytest.mark.parametrize("shape", SHAPES[-2:], ids=[s[0] for s in SHAPES[-2:]])
def test_zero_query_rows_on_a_replayable_plan(shape, kv):
    """As above, the prefill kernel reading the caches itself."""
    name, seq, n, hq, P = shape
    w = W.make_workload(22, seq, n, hq=hq, hkv=2, page_size=P, kv_dtype=kv, name=name, q_std=1e18,
                        softmax_scale=float(np.float32(0.07 / 1e18)))
    w.q[0] = 0
    run(w, replayable=True)


@pytest.mark.parametrize("kv", ["fp4", "fp8"])
@pytest.mark.parametrize("shape", SHAPES, ids=[s[0] for s in SHAPES])
def test_scales_whose_product_is_below_fp32(shape, kv):
    """softmax_scale * k_scale is zero in fp32 (both are positive): every score is
    as good as zero, and a masked one is still masked."""
    name, seq, n, hq, P = shape
    w = W.make_workload(23, seq, n, hq=hq, hkv=2, page_size=P, kv_dtype=kv, name=name, softmax_scale=1e-25)
    w.k_scale = 1e-25
    run(w)
