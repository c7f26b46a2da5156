"""attn_append_kv on 4-bit caches, attn_append_kv_rope and attn_read_kv through the
C ABI: caches and rotated queries bit for bit against the oracle's fp32 arithmetic."""
import numpy as np
import pytest

from asymmetric_kv_paged_gb300 import workloads as W
from oracle import append as A
from oracle import oracle

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def table(max_pos, rot):
    half = rot // 2
    inv = 10000.0 ** (-np.arange(half) / half)
    ang = np.arange(max_pos)[:, None] * inv
    return np.concatenate([np.cos(ang), np.sin(ang)], -1).astype(np.float32)


def rows(rng, *shape):
    return W.bf16_bits((rng.standard_normal(shape) * 2).astype(np.float32))


def dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits)).view(BF).cuda()


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF else torch.uint8).cpu().numpy().view(
        np.uint16 if t.dtype == BF else np.uint8)


def positions(w):
    return np.concatenate([np.arange(L - (b - a), L) for L, a, b in
                           zip(w.seq_lens, w.qo_indptr[:-1], w.qo_indptr[1:])]).astype(np.int64)


def setup(kv, seq, n, hq=16, hkv=2, P=16, dqk=192, seed=3, **kw):
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    w = W.make_workload(seed, seq, n, hq=hq, hkv=hkv, page_size=P, kv_dtype=kv, dqk=dqk, **kw)
    return w, DeviceWorkload(w)


def same_caches(dw, ref_k, ref_v):
    assert np.array_equal(bits(dw.k_cache).reshape(ref_k.shape), ref_k)
    assert np.array_equal(bits(dw.v_cache).reshape(ref_v.shape), ref_v)


CASES = [
    # name, kv, seq_lens, n, hq, hkv, P, dqk, rot, off, interleaved, given positions
    ("decode_bf16", "bf16", [1000, 129, 3000], [1, 1, 1], 16, 2, 128, 192, 64, 0, False, False),
    ("decode_fp4", "fp4", [1000, 1, 3000], [1, 1, 1], 16, 2, 128, 192, 64, 0, False, False),
    ("verify_fp8_pairs", "fp8", [700, 40], [8, 8], 16, 2, 16, 192, 64, 128, True, False),
    ("verify_fp4_pairs", "fp4", [700, 40], [8, 8], 16, 2, 16, 192, 64, 128, True, True),
    ("chunk_p1_whole", "fp4", [300], [120], 8, 1, 1, 192, 192, 0, False, False),
    ("chunk_p3_odd_half", "fp4", [260], [133], 16, 4, 3, 192, 48, 8, False, True),
    ("chunk_bf16_odd_half", "bf16", [260], [133], 16, 4, 3, 192, 16, 168, False, False),
    ("ragged_empty", "fp8", [90, 50, 20], [5, 0, 3], 8, 2, 3, 192, 112, 40, False, False),
    ("sym_fp4", "fp4", [90, 50, 20], [5, 0, 3], 8, 2, 64, 128, 128, 0, True, False),
    ("sym_bf16_g5", "bf16", [90, 33], [1, 33], 15, 3, 8, 128, 80, 48, False, False),
    ("many_requests", "fp4", [9] * 700, [1] * 700, 4, 1, 4, 192, 64, 0, False, False),
    ("a_warp_of_requests", "fp4", list(range(3, 35)), [1, 3] * 16, 8, 2, 16, 192, 64, 0, False, False),
    ("one_request_more", "bf16", list(range(3, 36)), [3, 1] * 16 + [2], 8, 2, 16, 192, 64, 64, True, False),
    ("tokens_past_the_warps_fp4", "fp4", [2999, 3000, 7, 1], [2400, 2470, 0, 1], 2, 1, 16, 192, 64, 0, False, False),
    ("tokens_past_the_warps_fp8", "fp8", [3000, 5, 2999], [2400, 4, 2500], 3, 1, 1, 128, 64, 64, True, True),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", CASES, ids=[c[0] for c in CASES])
def test_rotating_append_bit_exact(case, in_place):
    from asymmetric_kv_paged_gb300 import binding as B
    name, kv, seq, n, hq, hkv, P, dqk, rot, off, inter, given = case
    w, dw = setup(kv, seq, n, hq, hkv, P, dqk)
    rng = np.random.default_rng(7)
    kn, vn = rows(rng, w.total_q, hkv, dqk), rows(rng, w.total_q, hkv, 128)
    tab = table(3100, rot)
    pos = rng.integers(0, 3100, w.total_q) if given else positions(w)
    ks, vs = (0.0173, 0.0091) if kv == "fp4" else (w.k_scale, w.v_scale)
    cs = tab[pos][:, None]
    k_rot = A.rotate(W.bf16_values(kn), cs, rot, off, inter)
    ref_k, ref_v = A.append_rows(k_rot, W.bf16_values(vn), w.k_cache, w.v_cache, w.page_table, w.seq_lens,
                                 w.qo_indptr, kv, ks, vs)
    ref_q = A.f32_to_bf16(A.rotate(W.bf16_values(w.q), cs, rot, off, inter))
    rope = B.make_rope(torch.from_numpy(tab).cuda(), rot, off, inter,
                       torch.from_numpy(pos.astype(np.int32)).cuda() if given else None)
    q_out = dw.q if in_place else torch.full_like(dw.q, float("nan"))
    B.attn_append_kv_rope(dw.plan, rope, dw.q, dev(kn), dev(vn), q_out, dw.k_cache, dw.v_cache,
                          dw.page_table, dw.seq_lens, dw.qo_indptr, ks, vs)
    torch.cuda.synchronize()
    assert B.attn_get_device_error(dw.plan) == 0
    same_caches(dw, ref_k, ref_v)
    assert np.array_equal(bits(q_out), ref_q)


@pytest.mark.parametrize("P,dqk", [(16, 192), (1, 192), (128, 128)])
def test_fp4_append_bit_exact(P, dqk):
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup("fp4", [300, 77, 9], [130, 1, 9], P=P, dqk=dqk)
    rng = np.random.default_rng(11)
    k = (rng.standard_normal((w.total_q, 2, dqk)) * np.exp(rng.uniform(-14, 9, (w.total_q, 2, 1)))).astype(np.float32)
    v = rng.standard_normal((w.total_q, 2, 128)).astype(np.float32)
    k[0], v[1] = 0, -0.0
    k[2, 0, :16] = np.inf                                # saturates
    k[3, 0, 16:32] = np.repeat([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 2)     # ties under scale 1
    kn, vn = W.bf16_bits(k), W.bf16_bits(v)
    ref_k, ref_v = A.append_rows(W.bf16_values(kn), W.bf16_values(vn), w.k_cache, w.v_cache, w.page_table,
                                 w.seq_lens, w.qo_indptr, "fp4", 1.0, 0.013)
    B.attn_append_kv(dw.plan, dev(kn), dev(vn), dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens,
                     dw.qo_indptr, 1.0, 0.013)
    torch.cuda.synchronize()
    assert B.attn_get_device_error(dw.plan) == 0
    same_caches(dw, ref_k, ref_v)


def test_nan_makes_its_block_nan_and_no_other():
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup("fp4", [40], [2], hq=8, hkv=1)
    rng = np.random.default_rng(1)
    kn, vn = rows(rng, 2, 1, 192), rows(rng, 2, 1, 128)
    kn[0, 0, 37] = 0x7FC0
    B.attn_append_kv(dw.plan, dev(kn), dev(vn), dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens, dw.qo_indptr)
    ko, vo = torch.empty(2, 1, 192, dtype=BF, device="cuda"), torch.empty(2, 1, 128, dtype=BF, device="cuda")
    B.attn_read_kv(dw.plan, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens, dw.qo_indptr, ko, vo)
    nan = torch.isnan(ko).cpu().numpy()
    want = np.zeros_like(nan)
    want[0, 0, 32:48] = True
    assert np.array_equal(nan, want) and not torch.isnan(vo).any()


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("P,dqk,hkv", [(16, 192, 2), (1, 128, 3), (128, 192, 1)])
def test_read_returns_the_values_the_cache_holds(kv, P, dqk, hkv):
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup(kv, [300, 77, 9], [1, 1, 1], hq=hkv, hkv=hkv, P=P, dqk=dqk)
    ks, vs = (1.0, 1.0) if kv == "bf16" else (w.k_scale, 0.37)
    for counts in ([300, 77, 9], [3, 0, 9], [0, 64, 1]):
        ind = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
        T = int(ind[-1])
        ko = torch.full((T, hkv, dqk), 7.0, dtype=BF, device="cuda")
        vo = torch.full((T, hkv, 128), 7.0, dtype=BF, device="cuda")
        B.attn_read_kv(dw.plan, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens,
                       torch.from_numpy(ind).cuda(), ko, vo, ks, vs)
        pos = np.concatenate([np.arange(L - c, L) for L, c in zip(w.seq_lens, counts)])
        req = np.repeat(np.arange(3), counts)
        slot = w.page_table[req, pos // P].astype(np.int64) * P + pos % P
        for cache, out, d, sc in ((w.k_cache, ko, dqk, ks), (w.v_cache, vo, 128, vs)):
            r = cache.reshape(-1, hkv, cache.shape[-1])[slot]
            if kv == "bf16":
                want = r
            elif kv == "fp8":
                t = torch.from_numpy(r.copy()).view(torch.float8_e4m3fn).float().numpy()
                want = A.f32_to_bf16(t * np.float32(sc))
            else:
                want = A.f32_to_bf16(W.fp4_values(r, d) * np.float32(sc))
            assert np.array_equal(bits(out), want), (kv, counts)
    assert B.attn_get_device_error(dw.plan) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_bad_pages_positions_and_lengths_are_skipped(kv):
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup(kv, [60, 50, 40], [2, 1, 3], hq=8, hkv=2, P=16)
    rng = np.random.default_rng(2)
    kn, vn = rows(rng, 6, 2, 192), rows(rng, 6, 2, 128)
    tab = table(58, 64)                      # token 1 of request 0 is at 59: outside
    pt = dw.page_table.clone()
    pt[1, 49 // 16] = -1                     # request 1's new token: no such page
    lens = dw.seq_lens.clone()
    lens[2] = 2                              # request 2's first new token is at -1
    rope = B.make_rope(torch.from_numpy(tab).cuda(), 64, 0, False,
                       torch.tensor([57, 59, 49, 0, 1, 2], dtype=torch.int32, device="cuda"))
    q_out = torch.zeros_like(dw.q)
    before_k, before_v = bits(dw.k_cache).copy(), bits(dw.v_cache).copy()
    B.attn_append_kv_rope(dw.plan, rope, dw.q, dev(kn), dev(vn), q_out, dw.k_cache, dw.v_cache, pt, lens,
                          dw.qo_indptr, w.k_scale, w.v_scale)
    torch.cuda.synchronize()
    assert B.attn_get_device_error(dw.plan) == 1 | 4 | 8
    changed = (bits(dw.k_cache) != before_k).reshape(-1, 2 * before_k.shape[-1]).any(-1)
    table_ = w.page_table
    want = {int(table_[0, 58 // 16]) * 16 + 58 % 16, int(table_[2, 0]) * 16 + 0, int(table_[2, 0]) * 16 + 1}
    assert set(np.flatnonzero(changed).tolist()) == want
    changed = (bits(dw.v_cache) != before_v).reshape(-1, 2 * before_v.shape[-1]).any(-1)
    assert set(np.flatnonzero(changed).tolist()) == want
    written = (bits(q_out) != 0).any((1, 2))
    assert written.tolist() == [True, False, True, True, True, True]
    # reading the same rows: zeros where there is nothing to read
    ko = torch.full((8, 2, 192), 7.0, dtype=BF, device="cuda")
    vo = torch.full((8, 2, 128), 7.0, dtype=BF, device="cuda")
    B.attn_read_kv(dw.plan, dw.k_cache, dw.v_cache, pt, lens, dw.qo_indptr, ko, vo, w.k_scale, w.v_scale)
    assert B.attn_get_device_error(dw.plan) == 1 | 4
    zero = (bits(ko) == 0).all((1, 2)) & (bits(vo) == 0).all((1, 2))
    # rows: bad page; position -1; two rows past kv_indptr's last
    assert zero.tolist() == [False, False, True, True, False, False, True, True]


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_tokens_that_the_layout_does_not_hold_are_skipped(kv):
    """The device's qo_indptr ends two tokens early: those are reported, nothing of them
    is written, the others as ever."""
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup(kv, [60, 50], [4, 3], hq=8, hkv=2, P=16)
    rng = np.random.default_rng(4)
    kn, vn = rows(rng, 7, 2, 192), rows(rng, 7, 2, 128)
    tab = table(64, 64)
    rope = B.make_rope(torch.from_numpy(tab).cuda(), 64, 0, False)
    short = torch.tensor([0, 4, 5], dtype=torch.int32, device="cuda")
    lens = np.array([60, 50])
    pos = np.array([56, 57, 58, 59, 49])
    k_rot = A.rotate(W.bf16_values(kn[:5]), tab[pos][:, None], 64, 0, False)
    ref_k, ref_v = A.append_rows(k_rot, W.bf16_values(vn[:5]), w.k_cache, w.v_cache, w.page_table, lens,
                                 np.array([0, 4, 5]), kv, w.k_scale, w.v_scale)
    q_out = torch.zeros_like(dw.q)
    B.attn_append_kv_rope(dw.plan, rope, dw.q, dev(kn), dev(vn), q_out, dw.k_cache, dw.v_cache, dw.page_table,
                          dw.seq_lens, short, w.k_scale, w.v_scale)
    torch.cuda.synchronize()
    assert B.attn_get_device_error(dw.plan) == 4
    same_caches(dw, ref_k, ref_v)
    assert (bits(q_out) != 0).any((1, 2)).tolist() == [True] * 5 + [False] * 2


def test_refusals():
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup("fp4", [60], [2], hq=8, hkv=2, P=16)
    rng = np.random.default_rng(2)
    kn, vn = dev(rows(rng, 2, 2, 192)), dev(rows(rng, 2, 2, 128))
    tab = torch.from_numpy(table(100, 192)).cuda()
    before = bits(dw.k_cache).copy()

    def call(rot=64, off=0, cs=tab, q=dw.q, q_out=dw.q, k=kn, kc=dw.k_cache, ks=1.0, pt=dw.page_table):
        rope = B.attn_rope_t(cs.data_ptr(), None, cs.shape[0], rot, off, 0)
        B.attn_append_kv_rope(dw.plan, rope, q, k, vn, q_out, kc, dw.v_cache, pt, dw.seq_lens, dw.qo_indptr,
                              ks, 1.0)

    I, S = B.ATTN_ERR_INVALID_ARG, B.ATTN_ERR_UNSUPPORTED
    for kw, status in ((dict(rot=24), S), (dict(rot=64, off=4), S), (dict(rot=0), I), (dict(rot=-16), I),
                       (dict(rot=64, off=136), I), (dict(off=-8), I), (dict(q=None), I), (dict(q_out=None), I),
                       (dict(k=None), I), (dict(kc=None), I), (dict(pt=None), I), (dict(ks=0.0), I),
                       (dict(ks=float("nan")), I), (dict(ks=float("inf")), I), (dict(cs=tab[:0]), I),
                       (dict(cs=tab.view(-1)[1:192 * 50 + 1].view(50, 192)), I),
                       (dict(k=torch.empty(2 * 2 * 192 + 8, dtype=BF, device="cuda")[4:]), I)):
        with pytest.raises(B.AttnError) as e:
            call(**kw)
        assert e.value.status == status, kw
    ko = torch.empty(2 * 2 * 192 + 8, dtype=BF, device="cuda")
    for args in ((None, vn), (ko[4:-4].view(2, 2, 192), vn)):
        with pytest.raises((B.AttnError, AttributeError)):
            B.attn_read_kv(dw.plan, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens, dw.qo_indptr, *args)
    with pytest.raises(B.AttnError):
        B.attn_append_kv(dw.plan, kn, vn, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens, dw.qo_indptr, -1.0)
    torch.cuda.synchronize()
    assert np.array_equal(bits(dw.k_cache), before)
    call(q=None, q_out=None)                 # keys alone are fine
    torch.cuda.synchronize()
    assert B.attn_get_device_error(dw.plan) == 0


def test_no_tokens_is_no_work():
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup("fp4", [60, 9], [0, 0], hq=8, hkv=2, P=16)
    rope = B.make_rope(torch.from_numpy(table(100, 64)).cuda(), 64)
    e = torch.empty(0, 2, 192, dtype=BF, device="cuda")
    B.attn_append_kv_rope(dw.plan, rope, None, e, e, None, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens,
                          dw.qo_indptr)
    B.attn_read_kv(dw.plan, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens, dw.qo_indptr, e, e)
    torch.cuda.synchronize()
    assert B.attn_get_device_error(dw.plan) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_serving_steps_rotate_append_attend_in_one_graph(kv):
    """Decode steps as a server runs them: a replayable plan, one captured graph of the
    rotating append (queries in place), the device planner, attention and merge;
    lengths, projections and positions change between replays.  Every step's output is the
    oracle's on the oracle's own rotated and appended cache."""
    from asymmetric_kv_paged_gb300 import binding as B
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    steps = 3
    base = np.array([700, 300, 2000, 65], np.int64)
    g = W.make_workload(43, base + steps, [1, 1, 1, 1], hq=16, hkv=2, page_size=16, kv_dtype=kv, sinks=True)
    dw = DeviceWorkload(g, replayable=True)
    tab = table(2100, 64)
    rope = B.make_rope(torch.from_numpy(tab).cuda(), 64, 128, True)
    rng = np.random.default_rng(5)
    q, kn, vn = dw.q, dev(rows(rng, 4, 2, 192)), dev(rows(rng, 4, 2, 128))

    def step():
        B.attn_append_kv_rope(dw.plan, rope, q, kn, vn, q, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens,
                              dw.qo_indptr, g.k_scale, g.v_scale)
        dw.run()

    k_before, v_before = dw.k_cache.clone(), dw.v_cache.clone()
    dw.seq_lens.copy_(torch.from_numpy((base + 1).astype(np.int32)))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    dw.k_cache.copy_(k_before)
    dw.v_cache.copy_(v_before)
    kc, vc = g.k_cache, g.v_cache
    for s in range(steps):
        lens = (base + 1 + s).astype(np.int32)
        qb, kb, vb = rows(rng, 4, 16, 192), rows(rng, 4, 2, 192), rows(rng, 4, 2, 128)
        q.copy_(dev(qb)), kn.copy_(dev(kb)), vn.copy_(dev(vb))
        dw.seq_lens.copy_(torch.from_numpy(lens))
        graph.replay()
        torch.cuda.synchronize()
        cs = tab[lens - 1][:, None]
        kc, vc = A.append_rows(A.rotate(W.bf16_values(kb), cs, 64, 128, True), W.bf16_values(vb), kc, vc,
                               g.page_table, lens, g.qo_indptr, kv, g.k_scale, g.v_scale)
        same_caches(dw, kc, vc)
        pb = g.host_arrays()
        pb["q"] = A.f32_to_bf16(A.rotate(W.bf16_values(qb), cs, 64, 128, True))
        assert np.array_equal(bits(q), pb["q"])
        pb["seq_lens"] = lens
        pb["k_cache"], pb["v_cache"] = kc, vc
        if kv == "fp4":
            pb["k_cache"], pb["v_cache"] = W.bf16_bits(W.fp4_values(kc, 192)), W.bf16_bits(W.fp4_values(vc, 128))
        ref, _ = oracle.attn_paged(pb)
        mag = dict(pb)
        mag["v_cache"] = pb["v_cache"] & (0x7F if kv == "fp8" else 0x7FFF)
        a, _ = oracle.attn_paged(mag)
        got = dw.out.float().cpu().numpy()
        # weights and result in bf16, and the fp32 scores (|s| up to ~30) as for large scores
        assert np.all(np.abs(got - ref) <= 2.0 ** -8 * (1.2 * a + np.abs(ref)) + 1e-9), s
    assert B.attn_get_device_error(dw.plan) == 0
