"""A NaN block scale in a V row of a 4-bit cache: the block's 16 output dims are NaN
for the rows that see the key, and nothing else changes, bit for bit.  The keys are
those that some rows of a block see and others do not: the new tokens' own (causal
edge) and the first ones of a window."""
import numpy as np
import pytest

from asymmetric_kv_paged_gb300 import workloads as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

SHAPES = [
    # name, seq_lens, n, hq, page size, query/key head dim
    ("rows8", [90, 41], [1, 1], 16, 16, 192),
    ("rows8_pairs", [90, 700], [4, 2], 4, 16, 192),
    ("rows16", [90, 9000], [2, 2], 16, 16, 192),
    ("rows16_p1", [90, 9000], [4, 3], 8, 1, 192),
    ("rows32_few_tiles", [300, 66], [4, 3], 16, 16, 192),
    ("rows32_long", [16000, 66], [4, 4], 16, 128, 192),
    ("rows32_long_p3_d128", [16000, 66], [4, 1], 16, 3, 128),
    ("rows64", [330, 72], [8, 5], 16, 128, 192),
    ("rows64_p1", [330, 8], [8, 8], 16, 1, 192),
    ("rows64_long_d128", [9000, 64], [8, 8], 16, 16, 128),
    ("rows64_mixed", [700, 700, 260], [1, 8, 3], 16, 16, 192),
    ("rows128", [333, 65], [16, 2], 16, 16, 192),
    ("rows128_long_copies", [30000, 31000], [16, 2], 16, 128, 192),
    ("rows128_p3_d128", [500, 129], [15, 16], 16, 3, 128),
    ("rows128_chunk_d128", [500, 129], [300, 129], 16, 64, 128),
    ("rows256", [300, 200], [200, 200], 16, 16, 192),
    ("rows256_p1", [1000, 64], [130, 64], 16, 1, 192),
    ("rows256_long", [9000, 64], [300, 1], 16, 128, 192),
]


def events(w, rng):
    """(request, key, KV head, block) of the NaN scales: keys at the edges of what the
    new tokens see, one deep inside, and one that only the last token sees."""
    out = []
    for b in range(w.batch):
        L, n = int(w.seq_lens[b]), int(w.qo_indptr[b + 1] - w.qo_indptr[b])
        first = max(0, L - n - w.window + 1) if w.window else 0
        keys = {L - 1, L - n, L - n + n // 2, first, first + min(n, L - 1 - first) // 2, (first + L) // 2}
        for key in sorted(keys):
            out.append((b, key, int(rng.integers(2)), int(rng.integers(8))))
    return out


def expect(w, evs, hq):
    hit = np.zeros((w.total_q, hq, 128), bool)
    for b, key, g, blk in evs:
        t0, t1 = int(w.qo_indptr[b]), int(w.qo_indptr[b + 1])
        i = int(w.seq_lens[b]) - (t1 - t0) + np.arange(t1 - t0)
        see = (key <= i) & ((key > i - w.window) if w.window else True)
        hit[t0:t1][see, g * (hq // 2):(g + 1) * (hq // 2), 16 * blk:16 * blk + 16] = True
    return hit


def poison(w, evs):
    P = w.page_size
    v = w.v_cache.reshape(-1, 2, 80)
    for k, (b, key, g, blk) in enumerate(evs):
        slot = int(w.page_table[b, key // P]) * P + key % P
        v[slot, g, 64 + blk] = 0x7F if k % 2 else 0xFF


def outputs(dw):
    from asymmetric_kv_paged_gb300 import binding as B
    torch.cuda.synchronize()
    assert B.attn_get_device_error(dw.plan) == 0
    return dw.out.float().cpu().numpy(), dw.lse.cpu().numpy()


def compare(w, evs, hq, got, lse, ref, ref_lse):
    hit = expect(w, evs, hq)
    nan = np.isnan(got)
    assert np.array_equal(nan, hit), \
        f"{np.count_nonzero(nan & ~hit)} NaN too many, {np.count_nonzero(hit & ~nan)} missing of {hit.sum()}"
    assert np.array_equal(got[~hit], ref[~hit]) and np.array_equal(lse, ref_lse)


@pytest.mark.parametrize("window", [0, 1, 37])
@pytest.mark.parametrize("shape", SHAPES, ids=[s[0] for s in SHAPES])
def test_nan_value_block_reaches_the_rows_that_see_it(shape, window):
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    name, seq, n, hq, P, dqk = shape
    w = W.make_workload(31, seq, n, hq=hq, hkv=2, page_size=P, kv_dtype="fp4", window=window, sinks=window > 0,
                        name=name, dqk=dqk)
    clean = DeviceWorkload(w)
    clean.run()
    ref, ref_lse = outputs(clean)
    assert np.isfinite(ref).all()
    evs = events(w, np.random.default_rng(7))
    poison(w, evs)
    dw = DeviceWorkload(w)
    dw.run()
    got, lse = outputs(dw)
    compare(w, evs, hq, got, lse, ref, ref_lse)
    # a second run of the same plan on the clean cache is clean again
    dw.v_cache.copy_(clean.v_cache)
    dw.run()
    got, lse = outputs(dw)
    assert np.array_equal(got, ref) and np.array_equal(lse, ref_lse)


@pytest.mark.parametrize("window", [0, 37])
@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] in ("rows16", "rows64", "rows128", "rows256", "rows256_long")],
                         ids=lambda s: s[0])
def test_nan_value_block_on_a_replayable_plan(shape, window):
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    name, seq, n, hq, P, dqk = shape
    w = W.make_workload(32, seq, n, hq=hq, hkv=2, page_size=P, kv_dtype="fp4", window=window, name=name, dqk=dqk)
    dw = DeviceWorkload(w, replayable=True)
    dw.run()
    ref, ref_lse = outputs(dw)
    assert np.isfinite(ref).all()
    evs = events(w, np.random.default_rng(8))
    poison(w, evs)
    dw.v_cache.copy_(torch.from_numpy(w.v_cache))
    dw.run()
    got, lse = outputs(dw)
    compare(w, evs, hq, got, lse, ref, ref_lse)


@pytest.mark.parametrize("shape", [s for s in SHAPES if s[0] in ("rows64", "rows256", "rows256_p1")],
                         ids=lambda s: s[0])
def test_nan_value_block_without_a_workspace(shape):
    from asymmetric_kv_paged_gb300 import binding as B
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    name, seq, n, hq, P, dqk = shape
    w = W.make_workload(33, seq, n, hq=hq, hkv=2, page_size=P, kv_dtype="fp4", name=name, dqk=dqk)
    dw = DeviceWorkload(w)

    def run():
        B.attn_run_paged_no_workspace(dw.plan, dw.q, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens, dw.qo_indptr,
                                      None, 0, w.softmax_scale, w.k_scale, w.v_scale, dw.out, dw.lse)
        return outputs(dw)

    ref, ref_lse = run()
    evs = events(w, np.random.default_rng(9))
    poison(w, evs)
    dw.v_cache.copy_(torch.from_numpy(w.v_cache))
    compare(w, evs, hq, *run(), ref, ref_lse)


@pytest.mark.parametrize("value", [0x7FC0, 0x7F80, 0xFF80], ids=["nan", "inf", "-inf"])
@pytest.mark.parametrize("shape", SHAPES, ids=[s[0] for s in SHAPES])
def test_a_query_that_is_not_finite_stays_in_its_row(shape, value):
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    name, seq, n, hq, P, dqk = shape
    w = W.make_workload(34, seq, n, hq=hq, hkv=2, page_size=P, kv_dtype="fp4", name=name, dqk=dqk)
    clean = DeviceWorkload(w)
    clean.run()
    ref, ref_lse = outputs(clean)
    hit = np.zeros((w.total_q, hq), bool)
    for t, h, d in ((0, 1, 5), (w.total_q - 1, hq - 1, dqk - 1), (w.total_q // 2, 0, 64)):
        w.q[t, h, d] = value
        hit[t, h] = True
    dw = DeviceWorkload(w)
    dw.run()
    got, lse = outputs(dw)
    if value == 0x7FC0:
        assert np.all(np.isnan(got[hit])) and np.all(np.isnan(lse[hit]))
    assert np.array_equal(got[~hit], ref[~hit]) and np.array_equal(lse[~hit], ref_lse[~hit])
