"""attn_run_sparse against a plain 64-bit form, and the whole step: append, bounds, lists,
attention."""
import numpy as np
import pytest

import sparse_plain as P_
from asymmetric_kv_paged_gb300 import workloads as W
from oracle import append as A

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def setup(kv, seq, n, hq, hkv, P, dqk=192, sinks=False, seed=5, replayable=False, **kw):
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    w = W.make_workload(seed, seq, n, hq=hq, hkv=hkv, page_size=P, kv_dtype=kv, dqk=dqk, sinks=sinks, **kw)
    return w, DeviceWorkload(w, replayable=replayable)


def device(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def random_lists(rng, w, block, take, own_too=True, seq_lens=None):
    """Ascending lists of random blocks, the own one last, shorter ones padded; some empty."""
    seq_lens = w.seq_lens if seq_lens is None else seq_lens
    out = np.full((w.total_q, w.hkv, take), -1, np.int32)
    for b in range(w.batch):
        t0, t1 = int(w.qo_indptr[b]), int(w.qo_indptr[b + 1])
        for tok in range(t0, t1):
            own = (int(seq_lens[b]) - t1 + tok) // block
            for g in range(w.hkv):
                c = rng.permutation(own + 1)[:rng.integers(0, take + 1)]
                if own_too and len(c) and own not in c:
                    c[0] = own
                out[tok, g, :len(c)] = np.sort(c)
    return out


def run(w, dw, lists, block, seq_lens=None, pt=None, q=None):
    from asymmetric_kv_paged_gb300 import binding as B
    out = torch.full((w.total_q + 1, w.hq, 128), 7.0, dtype=BF, device="cuda")
    lse = torch.full((w.total_q + 1, w.hq), 7.0, device="cuda")
    B.attn_run_sparse(dw.plan, B.make_sparse(block, lists.shape[-1], 0, 1), dw.q if q is None else q, dw.k_cache,
                      dw.v_cache, dw.page_table if pt is None else pt, dw.seq_lens if seq_lens is None else seq_lens,
                      dw.qo_indptr, device(lists), dw.sinks, w.softmax_scale, w.k_scale, w.v_scale,
                      out[:w.total_q], lse[:w.total_q])
    o, l = out.double().cpu().numpy(), lse.double().cpu().numpy()
    assert (o[w.total_q] == 7).all() and (l[w.total_q] == 7).all()
    return o[:w.total_q], l[:w.total_q]


CASES = [
    # kv, dqk, seq_lens, n, hq, hkv, P, block, take, sinks
    ("bf16", 192, [3000, 700, 64, 1], [1] * 4, 16, 2, 64, 64, 16, False),
    ("fp8", 192, [3000, 700, 64, 1], [1] * 4, 16, 2, 128, 64, 16, True),
    ("fp4", 192, [3000, 700, 64, 1], [1] * 4, 16, 2, 128, 128, 9, False),
    ("bf16", 128, [500, 33], [8, 3], 8, 1, 48, 16, 11, True),
    ("fp8", 128, [500, 33], [8, 3], 12, 3, 32, 32, 7, False),
    ("fp4", 128, [500, 33], [8, 3], 40, 2, 16, 16, 13, True),
    ("bf16", 192, [900], [333], 16, 4, 64, 64, 6, False),          # neighbouring units share tiles
    ("fp8", 192, [700, 20], [300, 20], 32, 4, 64, 32, 6, True),
    ("fp4", 192, [1000, 300], [260, 300], 64, 4, 128, 128, 4, False),
    ("bf16", 128, [400, 380, 9, 77], [150, 170, 9, 60], 40, 2, 128, 16, 9, True),     # units of several requests
    ("fp4", 128, [800], [700], 4, 4, 16, 16, 12, False),
    ("fp8", 128, [640], [640], 8, 2, 128, 128, 5, False),          # own blocks cut at every place
    ("bf16", 192, [9000], [1], 128, 1, 64, 64, 140, False),        # a long list over a cluster
    ("fp8", 192, [4096], [2], 5, 1, 16, 16, 256, False),
    ("bf16", 192, [300] * 90, [3] * 90, 16, 2, 32, 32, 5, False),
    # many requests of a token each, and a group of more rows than a tile: a warp a unit
    ("bf16", 192, [200 + i for i in range(330)], [1] * 330, 16, 2, 64, 64, 3, True),
    ("fp4", 128, [90 + i for i in range(700)], [1] * 700, 4, 1, 16, 16, 4, False),
    ("fp8", 192, [400], [120], 130, 1, 64, 64, 3, False),
    # several tiles of tokens, lists of every length, small blocks side by side in a tile
    ("bf16", 192, [1500], [700], 16, 1, 16, 16, 40, True),
    ("bf16", 128, [800, 650], [400, 600], 3, 1, 32, 32, 9, False),
    ("fp8", 192, [1200], [900], 96, 1, 128, 128, 4, True),
    ("fp4", 192, [900], [640], 1, 1, 64, 64, 6, False),
    ("bf16", 192, [2000], [700], 2, 2, 64, 64, 20, False),
]


@pytest.mark.parametrize("kv,dqk,seq,n,hq,hkv,P,block,take,sinks", CASES)
def test_against_the_plain_form(kv, dqk, seq, n, hq, hkv, P, block, take, sinks):
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup(kv, seq, n, hq, hkv, P, dqk, sinks)
    lists = random_lists(np.random.default_rng(3), w, block, take)
    o, l = run(w, dw, lists, block)
    assert B.attn_get_device_error(dw.plan) == 0
    P_.assert_close(o, l, P_.attend(w, w.q, block, lists, w.sinks), kv)


@pytest.mark.parametrize("n", [1, 300])
def test_a_list_is_a_set(n):
    """Order, repetitions and where the empty entries stand change no bit."""
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup("bf16", [4000], [n], 16, 2, 32)
    rng = np.random.default_rng(3)
    lists = np.full((n, 2, 256), -1, np.int32)
    lists[..., :40] = random_lists(rng, w, 32, 40)
    mixed = lists.copy()
    for tok in range(n):
        for g in range(2):
            c = lists[tok, g][lists[tok, g] >= 0]
            c = np.concatenate([c, c[::2], c[:1], [-1, -5] * 20])
            mixed[tok, g, :len(c)] = rng.permutation(c)
    o, l = run(w, dw, lists, 32)
    o2, l2 = run(w, dw, mixed, 32)
    assert np.array_equal(o, o2) and np.array_equal(l, l2)
    assert B.attn_get_device_error(dw.plan) == 0
    P_.assert_close(o, l, P_.attend(w, w.q, 32, lists), "bf16")


@pytest.mark.parametrize("n", [1, 300])
def test_blocks_past_the_own_one_are_left_out(n):
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup("fp8", [900], [n], 16, 2, 64)
    lists = random_lists(np.random.default_rng(3), w, 64, 6)
    far = np.concatenate([lists, np.full((n, 2, 1), 15, np.int32), np.full((n, 2, 1), 2 ** 31 - 1, np.int32)], -1)
    o, l = run(w, dw, far, 64)
    assert B.attn_get_device_error(dw.plan) == 16
    P_.assert_close(o, l, P_.attend(w, w.q, 64, lists), "fp8")


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("n", [2, 300])
@pytest.mark.parametrize("block", [16, 128])
def test_unseen_slots_do_not_matter(kv, n, block):
    """Keys that a token does not see, and those only its neighbours chose, may be NaN: no bit
    of its rows changes; among the 300 tokens, where rows beside a NaN are summed anew in
    another order, they stay where they were, as close to the 64-bit form as before (either
    order is within assert_close's bound of it: the bound adds up every step's error in magnitude
    and holds for any order)."""
    w, dw = setup(kv, [1000], [n], 16, 2, 128)
    rng = np.random.default_rng(3)
    lists = random_lists(rng, w, block, 5)
    last = (n - 1) // 2                                            # tokens up to here never see block 2
    lists[:last + 1][lists[:last + 1] == 2] = -1
    o, l = run(w, dw, lists, block)
    for cache in (dw.k_cache, dw.v_cache):
        flat = cache.view(-1, *cache.shape[2:])
        for c in [*range(2 * block, 3 * block), 999]:
            flat[int(P_.slots(w, 0, c))] = float("nan") if kv == "bf16" else 0x7F
    o2, l2 = run(w, dw, lists, block)
    same = slice(0, last + 1)
    if n == 2:
        assert np.array_equal(o[same], o2[same]) and np.array_equal(l[same], l2[same])
    ref = P_.attend(w, w.q, block, lists)                          # (of the caches without the NaNs)
    for got in ((o, l), (o2, l2)):
        P_.assert_close(got[0][same], got[1][same], [x[same] for x in ref], kv)
    sees = ((lists[last + 1:] == 2).any(-1)) | ((lists[last + 1:] == 999 // block).any(-1) &
                                                (np.arange(last + 1, n) == n - 1)[:, None])
    assert np.array_equal(np.isnan(l2[last + 1:]).reshape(-1, 2, 8).all(-1), sees)
    assert np.array_equal(np.isnan(l2[last + 1:]).reshape(-1, 2, 8).any(-1), sees)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("seq,n", [([700, 90], [3, 1]), ([650], [400])])
def test_all_blocks_are_full_attention(kv, seq, n):
    """With every block listed the rows are those of attn_run_paged, up to the order of sums."""
    w, dw = setup(kv, seq, n, 16, 2, 64, sinks=True)
    dw.run()
    take = 11
    lists = np.broadcast_to(np.arange(take, dtype=np.int32), (w.total_q, 2, take)).copy()
    for b in range(w.batch):
        t = np.arange(w.qo_indptr[b], w.qo_indptr[b + 1])
        own = (w.seq_lens[b] - w.qo_indptr[b + 1] + t) // 64
        lists[t] = np.where(lists[t] <= own[:, None, None], lists[t], -1)
    o, l = run(w, dw, lists, 64)
    ref = P_.attend(w, w.q, 64, lists, w.sinks)
    P_.assert_close(o, l, ref, kv)
    P_.assert_close(dw.out.double().cpu().numpy(), dw.lse.double().cpu().numpy(), ref, "bf16")


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("n", [1, 200])
def test_large_and_tiny_queries(kv, n):
    """Scores of a few hundred (one weight is all there is) and rows of zeros, of one value, of
    the smallest bf16."""
    w, dw = setup(kv, [900], [n], 16, 2, 64, q_std=20.0)
    q = w.q.copy()
    q[0, 0] = 0
    q[0, 1] = 0x0001
    q[0, 9, 1:] = 0
    dw.q.copy_(device(q.view(np.int16)).view(BF))
    lists = random_lists(np.random.default_rng(3), w, 64, 6)
    lists[0] = [0, 2, 3, 5, 7, 10 if n == 200 else 14]
    o, l = run(w, dw, lists, 64)
    P_.assert_close(o, l, P_.attend(w, q, 64, lists), kv)


@pytest.mark.parametrize("n", [1, 200])
def test_odd_query_rows_stay_in_their_rows(n):
    w, dw = setup("fp8", [900], [n], 16, 2, 64)
    lists = random_lists(np.random.default_rng(3), w, 64, 6)
    lists[n - 1] = [0, 2, 3, 5, 7, 14]
    o, l = run(w, dw, lists, 64)
    q = dw.q.clone()
    q[n - 1, 3, 5] = float("nan")
    o2, l2 = run(w, dw, lists, 64, q=q)
    assert np.isnan(o2[n - 1, 3]).all() and np.isnan(l2[n - 1, 3])
    o2[n - 1, 3], l2[n - 1, 3] = o[n - 1, 3], l[n - 1, 3]
    assert np.array_equal(o, o2) and np.array_equal(l, l2)


def test_lengths_are_clamped_and_bad_pages_read_as_zeros():
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup("bf16", [500, 200], [1, 2], 16, 2, 64, replayable=True)
    lens = np.array([300, 100], np.int32)
    lists = random_lists(np.random.default_rng(3), w, 64, 4, seq_lens=lens)
    o, l = run(w, dw, lists, 64, seq_lens=device(lens))
    P_.assert_close(o, l, P_.attend(w, w.q, 64, lists, seq_lens=lens), "bf16")
    assert B.attn_get_device_error(dw.plan) == 0
    none = np.full((3, 2, 4), -1, np.int32)
    o, l = run(w, dw, none, 64, seq_lens=device(np.array([9000, 0], np.int32)))
    assert B.attn_get_device_error(dw.plan) == 4 and not o.any() and np.isinf(l).all()
    pt = dw.page_table.clone()
    pt[0, 1] = -3
    lists[...] = -1
    lists[0, :, :2] = [1, 2]
    o, l = run(w, dw, lists, 64, pt=pt, seq_lens=device(lens))
    assert B.attn_get_device_error(dw.plan) == 1
    k, v = w.k_cache.copy(), w.v_cache.copy()
    k[w.page_table[0, 1]], v[w.page_table[0, 1]] = 0, 0
    P_.assert_close(o, l, P_.attend(w, w.q, 64, lists, seq_lens=lens, k_cache=k, v_cache=v), "bf16")


def test_refusals():
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup("fp8", [300], [2], 16, 2, 64)
    lists = device(np.zeros((2, 2, 4), np.int32))
    out = torch.zeros(2, 16, 128, dtype=BF, device="cuda")
    I, S = B.ATTN_ERR_INVALID_ARG, B.ATTN_ERR_UNSUPPORTED

    def call(block=64, q=dw.q, k=dw.k_cache, idx=lists, o=out, scale=1.0, ks=1.0, sinks=None, pt=dw.page_table):
        B.attn_run_sparse(dw.plan, B.make_sparse(block, 4), q, k, dw.v_cache, pt, dw.seq_lens, dw.qo_indptr, idx,
                          sinks, scale, ks, 1.0, o)

    for kw, status in ((dict(block=8), S), (dict(block=128), S), (dict(q=None), I), (dict(k=None), I),
                       (dict(o=None), I), (dict(pt=None), I), (dict(scale=0.0), I), (dict(scale=float("inf")), I),
                       (dict(ks=-1.0), I), (dict(ks=float("nan")), I),
                       (dict(sinks=torch.zeros(16, device="cuda")), I),
                       (dict(o=torch.zeros(2 * 16 * 128 + 8, dtype=BF, device="cuda")[4:]), I)):
        with pytest.raises(B.AttnError) as e:
            call(**kw)
        assert e.value.status == status, kw
    with pytest.raises(ValueError):
        call(idx=lists[:, :1])
    torch.cuda.synchronize()
    assert not out.any() and B.attn_get_device_error(dw.plan) == 0
    call()


def table(max_pos, rot):
    inv = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    ang = np.arange(max_pos)[:, None] * inv
    return np.concatenate([np.cos(ang), np.sin(ang)], -1).astype(np.float32)


@pytest.mark.parametrize("kv,n", [("bf16", 1), ("fp8", 5), ("fp4", 1)])
def test_serving_steps_in_one_graph(kv, n):
    """Steps as a server runs them, captured once on a stream of their own: the rotating append
    by positions of three axes (shifted), bounds, lists, attention; lengths, projections and
    shifts change between replays, and blocks are completed on the way."""
    from asymmetric_kv_paged_gb300 import binding as B
    steps, block, take = 4, 16, 5
    base = np.array([630, 303, 1998, 64], np.int64)
    w, dw = setup(kv, base + steps * n, [n] * 4, 16, 2, 32, sinks=True, replayable=True)
    T, row = 4 * n, B.attn_bounds_row_bytes(192)
    tab = table(2100, 64)
    axes = B.mrope_axes([8, 12, 12], in_turn=True)
    delta = torch.zeros(4, dtype=torch.int32, device="cuda")
    mrope = B.make_mrope(device(tab), 64, axes, position_delta=delta, rot_offset=128)
    sparse = B.make_sparse(block, take, 1, 2)
    kn, vn = torch.zeros(T, 2, 192, dtype=BF, device="cuda"), torch.zeros(T, 2, 128, dtype=BF, device="cuda")
    # bounds of the prompts' blocks
    bounds = torch.zeros(w.num_pages, 2, 2, row, dtype=torch.uint8, device="cuda")
    lens = base.astype(np.int32)
    ind = np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)
    B.attn_update_bounds(dw.plan, block, dw.k_cache, bounds, dw.page_table, device(lens), device(ind), int(ind[-1]))
    ref_b = P_.update_bounds(w, np.zeros(bounds.shape, np.uint8), block, w.k_cache, lens, ind)
    assert np.array_equal(bounds.cpu().numpy(), ref_b)
    idx = torch.zeros(T, 2, take, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros(T, 16, 128, dtype=BF, device="cuda"), torch.zeros(T, 16, device="cuda")

    def step():
        B.attn_append_kv_mrope(dw.plan, mrope, dw.q, kn, vn, dw.q, dw.k_cache, dw.v_cache, dw.page_table,
                               dw.seq_lens, dw.qo_indptr, w.k_scale, w.v_scale)
        B.attn_update_bounds(dw.plan, block, dw.k_cache, bounds, dw.page_table, dw.seq_lens, dw.qo_indptr, T)
        B.attn_select_blocks(dw.plan, sparse, dw.q, bounds, dw.page_table, dw.seq_lens, dw.qo_indptr, idx)
        B.attn_run_sparse(dw.plan, sparse, dw.q, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens, dw.qo_indptr,
                          idx, dw.sinks, w.softmax_scale, w.k_scale, w.v_scale, out, lse)

    state = [t.clone() for t in (dw.k_cache, dw.v_cache, bounds)]
    dw.seq_lens.copy_(device((base + n).astype(np.int32)))
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t, s in zip((dw.k_cache, dw.v_cache, bounds), state):
        t.copy_(s)
    rng = np.random.default_rng(5)
    kc, vc = w.k_cache, w.v_cache
    for s in range(steps):
        lens = (base + n * (s + 1)).astype(np.int32)
        shift = -rng.integers(0, 40, 4).astype(np.int32)
        qb, kb, vb = (W.bf16_bits(rng.standard_normal(x).astype(np.float32))
                      for x in ((T, 16, 192), (T, 2, 192), (T, 2, 128)))
        for t, x in ((dw.q, qb), (kn, kb), (vn, vb)):
            t.copy_(device(x.view(np.int16)).view(BF))
        dw.seq_lens.copy_(device(lens))
        delta.copy_(device(shift))
        graph.replay()
        torch.cuda.synchronize()
        pos = np.concatenate([np.arange(L - n, L) + d for L, d in zip(lens, shift)])
        cs = tab[pos][:, None]
        kc, vc = A.append_rows(A.rotate(W.bf16_values(kb), cs, 64, 128, False), W.bf16_values(vb), kc, vc,
                               w.page_table, lens, w.qo_indptr, kv, w.k_scale, w.v_scale)
        q = A.f32_to_bf16(A.rotate(W.bf16_values(qb), cs, 64, 128, False))
        ref_b = P_.update_bounds(w, ref_b, block, kc, lens, w.qo_indptr)
        assert np.array_equal(bounds.cpu().numpy(), ref_b), s
        lists = P_.select(w, q, ref_b, block, take, 1, 2, lens)
        assert np.array_equal(idx.cpu().numpy(), lists), s
        P_.assert_close(out.double().cpu().numpy(), lse.double().cpu().numpy(),
                        P_.attend(w, q, block, lists, w.sinks, lens, kc, vc), kv, f"step {s}")
    assert B.attn_get_device_error(dw.plan) == 0
