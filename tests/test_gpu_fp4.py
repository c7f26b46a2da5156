"""Attention over a 4-bit cache through the C ABI, against the FP64 oracle on the
bf16 values the cache's rows stand for (exact).

Tolerance, per output element: with A = sum_j w_j |v_j| (the oracle on |V|), the
weights P are rounded to bf16 at worst (2^-8 each: 2^-8 A), the result to bf16
(2^-8 |out|), and the scores' fp32 sums (192 products, |s| up to ~10: 192 * 2^-24
* 10 = 1.2e-4 on an exponent) and exp2's 2^-22 add at most 2^-8 A / 20.
"""
import numpy as np
import pytest

from asymmetric_kv_paged_gb300 import workloads as W
from oracle import append as A
from oracle import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -8


def device(w, **kw):
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    return DeviceWorkload(w, **kw)


def err_word(dw):
    from asymmetric_kv_paged_gb300 import binding as B
    return B.attn_get_device_error(dw.plan)


def check(pb, out, lse, what=""):
    """out, lse (torch) against the oracle on the problem `pb` (host arrays)."""
    ref, ref_lse = oracle.attn_paged(pb)
    mag = dict(pb)
    mag["v_cache"] = pb["v_cache"] & 0x7FFF
    a, _ = oracle.attn_paged(mag)
    got = out.float().cpu().numpy().astype(np.float64)
    assert np.all(np.isfinite(got)), f"{what}: non-finite output"
    tol = U * (1.05 * a + np.abs(ref)) + 1e-9
    worst = (np.abs(got - ref) / tol).max() if got.size else 0.0
    assert worst <= 1, f"{what}: {worst:.3g} of the tolerance"
    if lse is not None:
        got = lse.cpu().numpy()
        both = np.isfinite(ref_lse)
        assert np.array_equal(both, np.isfinite(got))
        assert np.abs(got[both] - ref_lse[both]).max(initial=0) <= 3e-4, what


def run_and_check(w, **kw):
    dw = device(w, **kw)
    dw.out.fill_(float("nan"))
    dw.run()
    torch.cuda.synchronize()
    check(w.host_arrays(), dw.out, dw.lse, w.name)
    assert err_word(dw) == 0
    return dw


CASES = [
    # name, seq_lens, n, hq, hkv, P, window, sinks, query/key head dim
    ("decode_g8_p16", [512], [1], 8, 1, 16, 0, False, 192),
    ("decode_one_key", [1, 2, 65], [1, 1, 1], 8, 1, 16, 0, True, 192),
    ("decode_ragged_p128", [1000, 129, 3000, 64, 700], [1] * 5, 16, 2, 128, 0, False, 192),
    ("decode_ragged_p3", [50, 333, 1], [1, 1, 1], 8, 2, 3, 0, False, 192),
    ("decode_p1", [777, 64, 63], [1, 1, 1], 16, 2, 1, 0, True, 192),
    ("decode_p8", [777, 64, 1301], [1, 1, 1], 16, 2, 8, 0, False, 192),
    ("decode_g1", [300, 77], [1, 1], 4, 4, 16, 0, False, 192),
    ("decode_g16", [900, 4100], [1, 1], 16, 1, 128, 0, True, 192),
    ("decode_g20", [900, 300], [1, 1], 40, 2, 64, 0, False, 192),
    ("decode_g5_d128", [900, 333], [1, 1], 10, 2, 32, 0, True, 128),
    ("decode_long_d128", [9000, 100], [1, 1], 16, 2, 128, 0, False, 128),
    ("decode_long", [40000], [1], 16, 2, 128, 0, False, 192),
    ("two_tokens", [700, 66], [2, 2], 16, 2, 16, 0, True, 192),
    ("verify_p1", [1000, 555], [8, 8], 16, 2, 1, 0, False, 192),
    ("verify_p128", [2000, 130], [8, 3], 16, 2, 128, 0, False, 192),
    ("verify_d128_p3", [600, 9], [8, 8], 16, 2, 3, 0, True, 128),
    ("verify_wide", [800], [12], 16, 2, 16, 0, False, 192),
    ("all_new", [8, 1, 17], [8, 1, 17], 16, 2, 16, 0, False, 192),
    ("no_queries_between", [90, 50, 20], [5, 0, 3], 8, 2, 16, 0, True, 192),
    ("swa_sinks_mixed", [700, 700, 260, 900], [1, 8, 8, 1], 16, 2, 128, 128, True, 192),
    ("swa_decode", [700, 5000, 100], [1, 1, 1], 16, 2, 16, 128, True, 192),
    ("window_one", [300], [8], 8, 1, 16, 1, True, 192),
    ("swa_small_window_p3", [400, 90], [8, 2], 8, 2, 3, 5, True, 192),
    # 17 to 32 rows, enough key tiles for the register kernel
    ("rows32_p128", [12000, 5000, 130], [4, 3, 4], 16, 2, 128, 0, True, 192),
    ("rows24_p1", [9000, 7000], [3, 2], 16, 2, 1, 0, False, 192),
    ("rows32_d128_p16", [15500], [4], 16, 2, 16, 0, True, 128),
    ("rows20_swa_p8", [700 + 37 * i for i in range(80)], [4, 1, 3, 2] * 20, 10, 2, 8, 200, True, 192),
    ("rows32_p3_one_head", [30000], [2], 16, 1, 3, 0, False, 192),
    ("prefill_g16", [700], [300], 32, 2, 128, 0, False, 192),
    ("prefill_p1", [500], [130], 16, 2, 1, 0, True, 192),
    ("prefill_swa_p16", [900, 40], [400, 40], 16, 2, 16, 77, True, 192),
    ("prefill_d128", [500], [300], 16, 2, 64, 0, False, 128),
    ("chunk_m128_p3", [333], [15], 16, 2, 3, 0, False, 192),
]


def build(case, seed=5, **kw):
    name, seq, n, hq, hkv, P, win, sinks, dqk = case
    return W.make_workload(seed, seq, n, hq=hq, hkv=hkv, page_size=P, window=win, sinks=sinks,
                           kv_dtype="fp4", name="fp4_" + name, dqk=dqk, **kw)


@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_parity(case):
    run_and_check(build(case))


@pytest.mark.parametrize("seed", range(32))
def test_random_shapes(seed):
    rng = np.random.default_rng(900 + seed)
    hkv = int(rng.integers(1, 5))
    B = int(rng.integers(1, 6))
    n = [int(rng.choice([0, 1, 1, 1, 2, 8, 40, 150])) for _ in range(B)]
    if seed % 2:
        n = [min(x, 1) for x in n]
    n[0] = max(n[0], 1)
    seq = [x + int(rng.integers(0, 1500)) for x in n]
    run_and_check(build((f"random{seed}", seq, n, hkv * int(rng.choice([1, 2, 3, 8, 16])), hkv,
                         int(rng.choice([1, 2, 5, 8, 16, 64, 128, 192])),
                         int(rng.choice([0, 0, 1, 33, 400])), bool(rng.random() < 0.5),
                         int(rng.choice([192, 192, 128]))), seed=seed))


@pytest.mark.parametrize("P", [16, 1])
@pytest.mark.parametrize("n,hq", [(1, 8), (8, 16), (16, 16), (200, 16)], ids=["decode", "verify", "wide", "prefill"])
def test_every_code_and_scale_widens_exactly(n, hq, P):
    """window = 1: every query sees its own key alone, so the output is its V row,
    bit for bit (a bf16 value), for every code under every finite scale."""
    scales = np.array([s for s in range(256) if s & 0x7F != 0x7F], np.uint8)
    B = max(1, 32 // n)                                             # 32 rows x 8 scales see them all
    w = W.make_workload(3, [max(n, 40)] * B, [n] * B, hq=hq, hkv=2, page_size=P, window=1,
                        kv_dtype="fp4", k_std=0.5, name="exact")
    codes = (np.arange(8) * 2 | (np.arange(8) * 2 + 1) << 4).astype(np.uint8)   # a block's sixteen codes
    v = w.v_cache.reshape(-1, 2, 80)
    v[..., :64] = np.tile(codes, 8)
    row = 0
    for b in range(B):
        for i in range(int(w.seq_lens[b]) - n, int(w.seq_lens[b])):
            slot = int(w.page_table[b, i // P]) * P + i % P
            v[slot, :, 64:72] = scales[(8 * row + np.arange(8)) % len(scales)]
            row += 1
    assert row >= 32
    w.k_scale = w.v_scale = 1.0
    dw = device(w)
    dw.run()
    torch.cuda.synchronize()
    want = W.fp4_values(v, 128)
    got = dw.out.float().cpu().numpy().reshape(w.batch, n, 2, hq // 2, 128)
    for b in range(w.batch):
        for t in range(n):
            i = int(w.seq_lens[b]) - n + t
            slot = int(w.page_table[b, i // P]) * P + i % P
            assert np.array_equal(got[b, t], np.repeat(want[slot][:, None], hq // 2, 1)), (b, t)
    assert err_word(dw) == 0


@pytest.mark.parametrize("n,hq,P", [(1, 8, 16), (1, 8, 1), (8, 16, 16), (16, 16, 3), (300, 16, 16)])
def test_nan_scale_is_nan_and_stays_where_it_is_seen(n, hq, P):
    """A NaN block scale of a visible V row: its 16 output dims are NaN for the heads
    of that KV head, everything else is as without it."""
    w = W.make_workload(8, [max(n, 90) + 20, 70 + n], [n, n], hq=hq, hkv=2, page_size=P, kv_dtype="fp4")
    clean = device(w)
    clean.run()
    slot = int(w.page_table[0, 7 // P]) * P + 7 % P          # key 7 of request 0: every query sees it
    w.v_cache.reshape(-1, 2, 80)[slot, 1, 64 + 3] = 0x7F
    dw = device(w)
    dw.run()
    torch.cuda.synchronize()
    got, ref = dw.out.float().cpu().numpy(), clean.out.float().cpu().numpy()
    hit = np.zeros(got.shape, bool)
    hit[:n, hq // 2:, 48:64] = True
    assert np.all(np.isnan(got[hit])) and np.array_equal(got[~hit], ref[~hit])


@pytest.mark.parametrize("P", [16, 1])
@pytest.mark.parametrize("n,hq,seq", [(1, 8, 90), (1, 8, 9000), (2, 16, 9000), (4, 16, 9000), (4, 16, 16000),
                                      (8, 16, 9000), (16, 16, 300),
                                      (16, 16, 9000), (200, 16, 300), (200, 16, 9000)])
def test_nan_scale_of_a_key(n, hq, seq, P):
    """A NaN block scale of a visible K row makes its score NaN: the rows of that KV
    head that see the key are NaN, all others as without it (blocks of 4 to 256 rows,
    whole and split)."""
    w = W.make_workload(9, [seq + n, 70 + n], [n, n], hq=hq, hkv=2, page_size=P, kv_dtype="fp4")
    clean = device(w)
    clean.run()
    key = seq - 1 + n // 2                                    # later queries see it, earlier ones do not
    slot = int(w.page_table[0, key // P]) * P + key % P
    w.k_cache.reshape(-1, 2, 112)[slot, 1, 96 + 5] = 0xFF
    dw = device(w)
    dw.run()
    torch.cuda.synchronize()
    got, ref = dw.out.float().cpu().numpy(), clean.out.float().cpu().numpy()
    lse, ref_lse = dw.lse.cpu().numpy(), clean.lse.cpu().numpy()
    hit = np.zeros(got.shape[:2], bool)
    hit[key - seq:n, hq // 2:] = True
    if key < seq:
        hit[:n, hq // 2:] = True
    assert hit.any() and np.all(np.isnan(got[hit])) and np.all(np.isnan(lse[hit]))
    assert np.array_equal(got[~hit], ref[~hit]) and np.array_equal(lse[~hit], ref_lse[~hit])
    assert err_word(dw) == 0


@pytest.mark.parametrize("sinks", [False, True])
@pytest.mark.parametrize("n,hq,seq", [(1, 8, 5), (1, 8, 9000), (2, 16, 9000), (4, 16, 9000), (4, 16, 16000),
                                      (8, 16, 9000), (16, 16, 100),
                                      (16, 16, 9000), (200, 16, 200), (200, 16, 9000)])
def test_rows_with_nan_scores_only(n, hq, seq, sinks):
    """Every key of one KV head of a request is NaN: those rows are NaN, not empty."""
    w = W.make_workload(10, [seq + n, 70 + n], [n, n], hq=hq, hkv=2, page_size=16, sinks=sinks, kv_dtype="fp4")
    clean = device(w)
    clean.run()
    for key in range(seq + n):
        slot = int(w.page_table[0, key // 16]) * 16 + key % 16
        w.k_cache.reshape(-1, 2, 112)[slot, 0, 96] = 0x7F
    dw = device(w)
    dw.run()
    torch.cuda.synchronize()
    got, ref = dw.out.float().cpu().numpy(), clean.out.float().cpu().numpy()
    hit = np.zeros(got.shape[:2], bool)
    hit[:n, :hq // 2] = True
    assert np.all(np.isnan(got[hit])) and np.all(np.isnan(dw.lse.cpu().numpy()[hit]))
    assert np.array_equal(got[~hit], ref[~hit])


def test_large_scores_and_long_tails():
    """Scores of hundreds: weights that differ by more than any 16-bit range, the
    maximum rising late, in one segment and across splits."""
    for n, L in ((1, 6000), (8, 3001), (260, 900)):
        w = W.make_workload(12, [L], [n], hq=16, hkv=2, page_size=16, kv_dtype="fp4", q_std=8.0, k_std=3.0)
        dw = device(w)
        dw.run()
        torch.cuda.synchronize()
        ref, ref_lse = oracle.attn_paged(w.host_arrays())
        got = dw.out.float().cpu().numpy()
        # |s| up to ~300: the fp32 score is off by up to 192 * 2^-24 * 300 = 3.4e-3
        mag = w.host_arrays()
        mag["v_cache"] = mag["v_cache"] & 0x7FFF
        a, _ = oracle.attn_paged(mag)
        # prefill plans hold P in fp16: below 2^-14 of the running maximum it is a
        # multiple of 2^-24, off by 2^-25 at most for each of the L keys, and the
        # denominator is at least 1
        vmax = W.FP4_TOP * w.v_scale
        floor = L * 2.0 ** -25 * vmax if n == 260 else 0.0
        bad = np.abs(got - ref) > U * (a + np.abs(ref)) + 7e-3 * a + floor + 1e-9
        assert not bad.any(), (n, bad.sum())
        assert np.abs(dw.lse.cpu().numpy() - ref_lse).max() <= 7e-3


@pytest.mark.parametrize("std", [1e-20, 1e18])
def test_query_range(std):
    """Queries far outside fp16's range keep their bf16 precision."""
    for n in (1, 8, 200):
        w = W.make_workload(14, [400], [n], hq=8, hkv=1, page_size=16, kv_dtype="fp4", q_std=std,
                            softmax_scale=float(np.float32(0.07 / std)))
        run_and_check(w)


def test_replayed_graph_follows_the_lengths():
    w = build(("replay", [900, 200, 3000], [1, 1, 1], 16, 2, 16, 0, True, 192))
    dw = device(w, replayable=True)
    dw.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dw.run()
    for lens in ([900, 200, 3000], [1, 64, 65], [333, 199, 2999]):
        dw.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        pb = w.host_arrays()
        pb["seq_lens"] = np.array(lens, np.int32)
        check(pb, dw.out, dw.lse, str(lens))
    assert err_word(dw) == 0


@pytest.mark.parametrize("n,seqs,runs", [
    (2, [900, 200, 3000], ([900, 200, 3000], [2, 64, 66], [333, 199, 2999])),
    (4, [12000, 5000, 130], ([12000, 5000, 130], [4, 4, 4], [11999, 64, 5], [65, 4999, 129])),
    (8, [900, 200], ([900, 200], [8, 8], [65, 199]))])
def test_replayed_graph_of_draft_tokens(n, seqs, runs):
    w = build(("replay_draft", seqs, [n] * len(seqs), 16, 2, 128, 0, True, 192))
    dw = device(w, replayable=True)
    dw.run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        dw.run()
    for lens in runs:
        dw.seq_lens.copy_(torch.tensor(lens, dtype=torch.int32))
        g.replay()
        torch.cuda.synchronize()
        pb = w.host_arrays()
        pb["seq_lens"] = np.array(lens, np.int32)
        check(pb, dw.out, dw.lse, str(lens))
    assert err_word(dw) == 0


@pytest.mark.parametrize("n,L", [(2, 6000), (4, 16000)])
def test_large_scores_of_draft_tokens(n, L):
    """As test_large_scores_and_long_tails, same tolerance, for 16 and 32 rows."""
    w = W.make_workload(13, [L], [n], hq=16, hkv=2, page_size=128, kv_dtype="fp4", q_std=8.0, k_std=3.0)
    dw = device(w)
    dw.run()
    torch.cuda.synchronize()
    ref, ref_lse = oracle.attn_paged(w.host_arrays())
    mag = w.host_arrays()
    mag["v_cache"] = mag["v_cache"] & 0x7FFF
    a, _ = oracle.attn_paged(mag)
    got = dw.out.float().cpu().numpy()
    assert np.all(np.abs(got - ref) <= U * (a + np.abs(ref)) + 7e-3 * a + 1e-9)
    assert np.abs(dw.lse.cpu().numpy() - ref_lse).max() <= 7e-3


@pytest.mark.parametrize("n", [8, 100])
def test_replayable_verify_and_prefill(n):
    w = build(("replayable", [900, 200], [n, n], 16, 2, 16, 0, False, 192))
    run_and_check(w, replayable=True)


@pytest.mark.parametrize("n", [1, 8, 100])
def test_no_workspace(n):
    from asymmetric_kv_paged_gb300 import binding as B
    w = build(("no_workspace", [2900, 200], [n, n], 16, 2, 16, 0, True, 192))
    dw = device(w)
    B.attn_run_paged_no_workspace(dw.plan, dw.q, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens,
                                  dw.qo_indptr, dw.sinks, w.window, w.softmax_scale, w.k_scale, w.v_scale,
                                  dw.out, dw.lse)
    torch.cuda.synchronize()
    check(w.host_arrays(), dw.out, dw.lse)
    assert err_word(dw) == 0


@pytest.mark.parametrize("n,P", [(1, 16), (1, 3), (8, 16), (100, 16)])
def test_bad_page_id_is_reported_and_read_as_zeros(n, P):
    w = W.make_workload(9, [400], [n], hq=8, hkv=1, page_size=P, kv_dtype="fp4")
    dw = device(w)
    dw.page_table[0, 5] = w.num_pages + 3
    dw.run()
    torch.cuda.synchronize()
    assert err_word(dw) == 1
    pb = w.host_arrays()
    page = int(w.page_table[0, 5])
    pb["k_cache"][page] = 0
    pb["v_cache"][page] = 0
    check(pb, dw.out, dw.lse)


def test_refusals():
    from asymmetric_kv_paged_gb300 import binding as B
    w = build(CASES[0])
    dw = device(w)

    def call(k=None, ks=1.0, vs=1.0, scale=0.1, ws=None, q=None):
        B.attn_run_paged(dw.plan, dw.q if q is None else q, dw.k_cache if k is None else k, dw.v_cache,
                         dw.page_table, dw.seq_lens, dw.qo_indptr, None, 0, scale, ks, vs, dw.out, dw.lse,
                         dw.workspace if ws is None else ws)

    spare = torch.empty(dw.k_cache.numel() + 16, dtype=torch.uint8, device="cuda")
    for kw in (dict(ks=0.0), dict(ks=-1.0), dict(ks=float("nan")), dict(vs=float("inf")), dict(scale=0.0),
               dict(k=spare[8:]), dict(q=dw.q.view(-1)[4:])):
        with pytest.raises(B.AttnError) as e:
            call(**kw)
        assert e.value.status == B.ATTN_ERR_INVALID_ARG, kw
    if dw.plan.workspace_bytes:
        with pytest.raises(B.AttnError) as e:
            call(ws=dw.workspace[:1])
        assert e.value.status == B.ATTN_ERR_WORKSPACE
    dw.run()
    torch.cuda.synchronize()
    check(w.host_arrays(), dw.out, dw.lse)


def test_other_stream():
    w = build(CASES[2])
    dw = device(w)
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    dw.run(stream=st)
    st.synchronize()
    check(w.host_arrays(), dw.out, dw.lse)


def test_offsets_past_32_bits():
    """A pool whose last rows lie more than 2^32 bytes in: the slots in use are at
    its end."""
    P, hkv = 128, 4
    pages = (1 << 32) // (P * hkv * 80) + 40             # V: over 2^32 bytes; K more
    w = W.make_workload(2, [300, 77], [1, 8], hq=32, hkv=hkv, page_size=P, kv_dtype="fp4")
    used = w.num_pages
    dw = device(w)
    kc = torch.full((pages, P, hkv, 112), 0xFF, dtype=torch.uint8, device="cuda")
    vc = torch.full((pages, P, hkv, 80), 0xFF, dtype=torch.uint8, device="cuda")
    kc[pages - used:], vc[pages - used:] = dw.k_cache, dw.v_cache
    from asymmetric_kv_paged_gb300 import binding as B
    prob, keep = dw.problem()
    prob.num_pages = pages
    plan = B.attn_plan(prob, 0, keep)
    B.attn_run_paged(plan, dw.q, kc, vc, dw.page_table + (pages - used), dw.seq_lens, dw.qo_indptr, None, 0,
                     w.softmax_scale, w.k_scale, w.v_scale, dw.out, dw.lse,
                     torch.empty(max(1, plan.workspace_bytes), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    check(w.host_arrays(), dw.out, dw.lse)


def test_oracle_values_of_the_device_cache_are_exact():
    """The bf16 the tests hand to the oracle is what the format's bit fields say."""
    w = build(CASES[3])
    k = W.bf16_values(w.host_arrays()["k_cache"])
    for slot in range(5):
        row = w.k_cache.reshape(-1, w.hkv, 112)[slot, 0]
        assert np.array_equal(k.reshape(-1, w.hkv, 192)[slot, 0], A.fp4_row_values(row, 192), equal_nan=True)
