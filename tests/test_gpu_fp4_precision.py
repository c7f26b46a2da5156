"""The weights of attention over a 4-bit cache keep fp16's 11 bits: cases in which a
coarser weight shows.

Every 32 keys (a unit of the kernels' work at the smallest) hold one key of score s
and 31 of score 0, whose weight is a chosen fraction of the heavy one's everywhere.

Tolerance per output element, A = sum_j w_j |v_j|: the weights' fp16 rounding, 2^-11
A; the scores are exact products (one nonzero query element), exp2 and the fp32 sums
of at most L / 16 partial products add less than 2^-13 A; the result's bf16 rounding,
2^-8 |out|.
"""
import numpy as np
import pytest

from asymmetric_kv_paged_gb300 import workloads as W
from oracle import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SHAPES = [
    # name, seq_lens, n, hq, page size, query/key head dim
    ("rows8", [2000, 1], [1, 1], 16, 16, 192),
    ("rows8_p1_d128", [2000, 33], [1, 1], 16, 1, 128),
    ("rows16", [2000, 300], [2, 2], 16, 128, 192),
    ("rows32_few_tiles", [2000], [4], 16, 16, 192),
    ("rows32_long", [16000], [4], 16, 16, 192),
    ("rows64", [2000, 90], [8, 8], 16, 16, 192),
    ("rows128", [2000, 16], [16, 16], 16, 3, 192),
    ("rows256", [2000, 200], [200, 100], 16, 16, 192),
]


def build(shape, fraction, light, heavy):
    """light, heavy: (code byte, scale byte) of the V rows' values."""
    name, seq, n, hq, P, dqk = shape
    w = W.make_workload(41, seq, n, hq=hq, hkv=2, page_size=P, kv_dtype="fp4", name=name, dqk=dqk,
                        softmax_scale=float(np.float32(-np.log(fraction))))
    w.k_scale = w.v_scale = 1.0
    w.q[:] = 0
    w.q[..., 0] = 0x3F80                              # 1
    kc, vc = w.k_cache.reshape(-1, 2, w.k_cache.shape[-1]), w.v_cache.reshape(-1, 2, 80)
    for b in range(w.batch):
        j = np.arange(int(w.seq_lens[b]))
        slot = w.page_table[b, j // P].astype(np.int64) * P + j % P
        kc[slot] = 0
        kc[slot, :, dqk // 2:dqk // 2 + dqk // 16] = 0x38           # scales of 1
        kc[slot[::32], :, 0] = 0x02                                 # dim 0 of a heavy key: 1
        for sl, (code, scale) in ((slot, light), (slot[::32], heavy)):
            vc[sl, :, :64] = code
            vc[sl, :, 64:72] = scale
    return w


def run(w, **kw):
    from asymmetric_kv_paged_gb300 import binding as B
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    dw = DeviceWorkload(w, **kw)
    dw.run()
    torch.cuda.synchronize()
    assert B.attn_get_device_error(dw.plan) == 0
    ref, _ = oracle.attn_paged(w.host_arrays())
    mag = w.host_arrays()
    mag["v_cache"] = mag["v_cache"] & 0x7FFF
    a, _ = oracle.attn_paged(mag)
    return dw.out.float().cpu().numpy().astype(np.float64), ref, a


def bf16_weights(w):
    """The output if the weights were rounded to bf16, for the last token (it sees
    whole units but for the last)."""
    L = int(w.seq_lens[0])
    heavy = np.arange(L) % 32 == 0
    p = np.where(heavy, 1.0, np.exp2(-np.log2(np.e) * w.softmax_scale))
    r = W.bf16_values(W.bf16_bits(p.astype(np.float32))).astype(np.float64)
    P = w.page_size
    j = np.arange(L)
    slot = w.page_table[0, j // P].astype(np.int64) * P + j % P
    v = W.fp4_values(w.v_cache.reshape(-1, 2, 80)[slot, 0], 128).astype(np.float64)[:, 0]
    return (r * v).sum() / p.sum(), (p * v).sum() / p.sum(), (p * np.abs(v)).sum() / p.sum()


@pytest.mark.parametrize("shape", SHAPES, ids=[s[0] for s in SHAPES])
def test_weights_that_cancel(shape):
    """Heavy values of -3.75 against 31 light ones of 0.5 with a quarter of the weight:
    the result is 1% of A.  A quarter times 1 + 2^-8 + 2^-12 lies between two bf16
    values, off by nearly 2^-8 of half of A."""
    w = build(shape, 0.25 * (1 + 2.0 ** -8 + 2.0 ** -12), (0x11, 0x38), (0xFF, 0x32))
    got, ref, a = run(w)
    assert np.all(np.abs(got - ref) <= (2.0 ** -11 + 2.0 ** -13) * a + 2.0 ** -8 * np.abs(ref))
    off, want, mag = bf16_weights(w)
    if w.seq_lens[0] >= 2000:                         # the case tells the two apart
        assert abs(off - want) > (2.0 ** -11 + 2.0 ** -13) * mag + 2.0 ** -8 * abs(want)


@pytest.mark.parametrize("shape", SHAPES, ids=[s[0] for s in SHAPES])
def test_small_weights(shape, **kw):
    """Light weights of 2^-20 (1 + 2^-5.1), heavy values of zero: the result is the
    light keys' alone.  Without the factor of 2^7 that the weights are held with, fp16
    would have steps of 2^-24 there, and the nearest one is 2^-5.1 off."""
    fraction = 2.0 ** -20 * (1 + 2.0 ** -5.1)
    w = build(shape, fraction, (0x66, 0x38), (0x00, 0x38))
    got, ref, a = run(w, **kw)
    bound = 2.0 ** -11 + 2.0 ** -13 + 2.0 ** -8              # the result is A
    assert np.all(np.abs(got - ref) <= bound * a)
    assert abs(float(np.float16(fraction)) / fraction - 1) > bound


def test_small_weights_on_a_replayable_plan():
    test_small_weights(SHAPES[-1], replayable=True)
