"""Attention over selected blocks where sizes, layouts and histories are unusual: several CTAs
a token tile, empty requests, steps of several tokens replayed from a graph with lists of every
kind, the longest requests, pools and bounds of more than 2^32 bytes."""
import numpy as np
import pytest

import sparse_plain as P_
from asymmetric_kv_paged_gb300 import workloads as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_select import device, random_bounds, run as select, setup as select_setup  # noqa: E402
from test_gpu_sparse import random_lists, run as attend, setup as sparse_setup  # noqa: E402

BF = torch.bfloat16


@pytest.mark.parametrize("n", [1, 200])
def test_queries_of_the_largest_magnitude(n):
    """127.5 * 2^121 and its neighbours: whole numbers of up to 128."""
    w, dw = select_setup([3000], [n], 16, 2, 64)
    rng = np.random.default_rng(4)
    bounds = random_bounds(rng, w, 64)
    q = rng.choice([0x7F7F, 0x7F7E, 0xFF7F, 0x7E7F, 0xFEC0], (n, 16, 192)).astype(np.uint16)
    assert np.array_equal(select(w, dw, q, bounds, 64, 9, 1, 1), P_.select(w, q, bounds, 64, 9, 1, 1))


@pytest.mark.parametrize("seq,n,hq,hkv,P,dqk,block,take", [
    ([13000], [90], 16, 4, 64, 192, 16, 24),                     # four CTAs share out 810 blocks
    ([33000], [96], 8, 4, 128, 128, 16, 9),                      # eight, 2,062 blocks, more than a warp holds
    ([20000, 300, 21000], [60, 40, 64], 32, 2, 16, 192, 16, 40),
])
def test_lists_of_a_chunk_over_clusters(seq, n, hq, hkv, P, dqk, block, take):
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = select_setup(seq, n, hq, hkv, P, dqk)
    bounds = random_bounds(np.random.default_rng(3), w, block)
    got = select(w, dw, w.q, bounds, block, take, 1, 2)
    assert B.attn_get_device_error(dw.plan) == 0
    assert np.array_equal(got, P_.select(w, w.q, bounds, block, take, 1, 2))


RAGGED = ([700, 1, 16, 900, 40, 333], [300, 0, 16, 0, 1, 333])
MANY = ([150 + 3 * i for i in range(40)], [20] * 40)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("seq,n", [RAGGED, MANY])
def test_chunks_of_ragged_batches(kv, seq, n):
    """Requests of no new token, of one, of whole and broken tiles, and more than 32 of them;
    lengths below the plan's."""
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = sparse_setup(kv, seq, n, 16, 2, 32, replayable=True)
    lens = np.maximum(np.asarray(n), np.asarray(seq) - 5).astype(np.int32)
    lists = random_lists(np.random.default_rng(3), w, 32, 6, seq_lens=lens)
    o, l = attend(w, dw, lists, 32, seq_lens=device(lens))
    P_.assert_close(o, l, P_.attend(w, w.q, 32, lists, seq_lens=lens), kv)
    bounds = random_bounds(np.random.default_rng(3), w, 32)
    got = select(w, dw, w.q, bounds, 32, 6, 1, 1, device(lens))
    assert np.array_equal(got, P_.select(w, w.q, bounds, 32, 6, 1, 1, lens))
    assert B.attn_get_device_error(dw.plan) == 0


@pytest.mark.parametrize("kv", ["bf16", "fp4"])
def test_a_chunk_replayed_with_lists_of_every_kind(kv):
    """One captured run over a chunk of tokens: ascending lists, then mixed ones, then lengths and
    lists anew, then ascending ones again; eager runs between the replays."""
    from asymmetric_kv_paged_gb300 import binding as B
    n, block, take = 300, 32, 12
    w, dw = sparse_setup(kv, [1000], [n], 16, 2, 64, replayable=True)
    rng = np.random.default_rng(8)
    idx = torch.zeros(n, 2, take, dtype=torch.int32, device="cuda")
    out, lse = torch.zeros(n, 16, 128, dtype=BF, device="cuda"), torch.zeros(n, 16, device="cuda")
    sparse = B.make_sparse(block, take)

    def call():
        B.attn_run_sparse(dw.plan, sparse, dw.q, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens, dw.qo_indptr,
                          idx, dw.sinks, w.softmax_scale, w.k_scale, w.v_scale, out, lse)

    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call()
    stream.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step, L in enumerate([1000, 1000, 640, 640, 1000]):
        lens = np.array([L], np.int32)
        lists = random_lists(rng, w, block, take, seq_lens=lens)
        if step & 1:
            lists = rng.permuted(lists, axis=-1)
        dw.seq_lens.copy_(device(lens))
        idx.copy_(device(lists))
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        ref = P_.attend(w, w.q, block, lists, seq_lens=lens)
        got = out.double().cpu().numpy(), lse.double().cpu().numpy()
        P_.assert_close(*got, ref, kv, f"step {step}")
        out.fill_(float("nan"))
        with torch.cuda.stream(stream):                          # eager, behind the replay
            call()
        stream.synchronize()
        assert np.array_equal(out.double().cpu().numpy(), got[0])
    assert B.attn_get_device_error(dw.plan) == 0


@pytest.mark.parametrize("seq,n", [([900], [2]), ([900], [300])])
def test_rows_that_the_layout_does_not_hold_stay(seq, n):
    """A device layout of fewer tokens than the plan's (against the rules): the rows behind it are
    left as they were, and bit 2 is set."""
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = sparse_setup("bf16", seq, n, 16, 2, 64)
    m = n[0] - 1
    dw.qo_indptr.copy_(device(np.array([0, m], np.int32)))
    lists = device(random_lists(np.random.default_rng(3), w, 64, 4))
    sparse = B.make_sparse(64, 4)
    out = torch.full((n[0], 16, 128), 7.0, dtype=BF, device="cuda")
    B.attn_run_sparse(dw.plan, sparse, dw.q, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens, dw.qo_indptr, lists,
                      None, w.softmax_scale, w.k_scale, w.v_scale, out)
    bounds = device(random_bounds(np.random.default_rng(3), w, 64))
    idx = torch.full((n[0], 2, 4), -7, dtype=torch.int32, device="cuda")
    B.attn_select_blocks(dw.plan, sparse, dw.q, bounds, dw.page_table, dw.seq_lens, dw.qo_indptr, idx)
    torch.cuda.synchronize()
    assert (out[m:] == 7).all() and (idx[m:] == -7).all()
    assert not (out[:m] == 7).all(-1).any() and (idx[:m] >= -1).all()
    assert n[0] > 16 or B.attn_get_device_error(dw.plan) == 4    # (whole tiles of rows may hide one)


def test_the_most_blocks():
    """A request of 49,152 blocks of 16, 256 of them taken; one block more is refused, and so are
    more query rows than the scores leave room for."""
    from asymmetric_kv_paged_gb300 import binding as B
    N = 49152
    rng = np.random.default_rng(2)
    rec = np.zeros((N, 1, 1, 272), np.int8)
    rec[..., :256] = rng.integers(-20, 21, (N, 1, 1, 256))
    rec[..., 128:256] = np.minimum(rec[..., :128], rec[..., 128:256])
    bounds = device(rec.view(np.uint8))
    table = rng.permutation(N).astype(np.int32)
    qb = W.bf16_bits(rng.standard_normal((1, 8, 128)).astype(np.float32))
    q = device(np.tile(qb, (1, 16, 1)).view(np.int16)).view(BF)
    ind = np.array([0, 1], np.int32)

    def call(hq, blocks):
        lens = np.array([16 * blocks], np.int32)
        prob, keep = B.make_problem(1, hq, 1, 16, N, blocks, B.ATTN_KV_BF16, 0, False, ind, lens, head_dim_qk=128)
        plan = B.attn_plan(prob, 0, keep)
        idx = torch.full((1, 1, 256), -7, dtype=torch.int32, device="cuda")
        B.attn_select_blocks(plan, B.make_sparse(16, 256, 1, 1), q[:, :hq].contiguous(), bounds,
                             device(np.resize(table, blocks)), device(lens), device(ind), idx)
        assert B.attn_get_device_error(plan) == 0
        return idx.cpu().numpy()[0, 0]

    s = P_.scores(W.bf16_values(qb[0]).astype(np.float64), rec[table, 0, 0].view(np.uint8), 128)
    assert np.array_equal(call(8, N), P_.choose(s, N - 1, 256, 1, 1))
    for hq, blocks in ((8, N + 1), (128, N)):
        with pytest.raises(B.AttnError) as e:
            call(hq, blocks)
        assert e.value.status == B.ATTN_ERR_UNSUPPORTED


@pytest.mark.parametrize("kv,n", [("bf16", 2), ("bf16", 200), ("fp8", 200), ("fp4", 2), ("fp4", 200)])
def test_attention_far_into_a_pool(kv, n):
    """The workload's pages at the end of caches of more than 2^32 bytes: the same bits."""
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = sparse_setup(kv, [700 + n, n], [n, n], 16, 2, 64)
    lists = random_lists(np.random.default_rng(3), w, 64, 5)
    o, l = attend(w, dw, lists, 64)
    page_bytes = dw.v_cache[0].numel() * dw.v_cache.element_size()
    pages = (1 << 32) // page_bytes + 2 * w.num_pages
    far = []
    for t in (dw.k_cache, dw.v_cache):
        big = torch.empty(pages, *t.shape[1:], dtype=t.dtype, device="cuda")
        big[pages - w.num_pages:] = t
        far.append(big)
    pt = dw.page_table + (pages - w.num_pages)
    prob, keep = dw.problem()
    prob.num_pages = pages
    plan = B.attn_plan(prob, 0, keep)
    out = torch.empty(w.total_q, 16, 128, dtype=BF, device="cuda")
    B.attn_run_sparse(plan, B.make_sparse(64, 5, 0, 1), dw.q, *far, pt, dw.seq_lens, dw.qo_indptr, device(lists), None,
                      w.softmax_scale, w.k_scale, w.v_scale, out)
    assert B.attn_get_device_error(plan) == 0
    assert np.array_equal(out.double().cpu().numpy(), o)
    del far, big
    torch.cuda.empty_cache()


@pytest.mark.parametrize("n", [3, 200])
def test_bounds_far_into_their_array(n):
    """Records more than 2^32 bytes in: written, read back and chosen by as in a small array."""
    from asymmetric_kv_paged_gb300 import binding as B
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    w = W.make_workload(5, [900, 300], [n, n], hq=32, hkv=8, page_size=16, kv_dtype="fp4")
    dw = DeviceWorkload(w)
    row = B.attn_bounds_row_bytes(192)
    pages = (1 << 32) // (8 * row) + 2 * w.num_pages
    prob, keep = dw.problem()
    prob.num_pages = pages
    plan = B.attn_plan(prob, 0, keep)
    k_far = torch.empty(pages, *dw.k_cache.shape[1:], dtype=torch.uint8, device="cuda")
    k_far[pages - w.num_pages:] = dw.k_cache
    sparse, got = B.make_sparse(16, 8, 1, 1), []
    ind = device(np.array([0, 900, 1200], np.int32))
    blocks = np.array([0, 900 // 16, 900 // 16 + 300 // 16], np.int32)
    for p, k, num, pt in ((dw.plan, dw.k_cache, w.num_pages, dw.page_table),
                          (plan, k_far, pages, dw.page_table + (pages - w.num_pages))):
        bounds = torch.empty(num, 1, 8, row, dtype=torch.uint8, device="cuda")
        B.attn_update_bounds(p, 16, k, bounds, pt, dw.seq_lens, ind, 1200)
        out = torch.empty(int(blocks[-1]), 8, 2, 192, dtype=BF, device="cuda")
        B.attn_read_bounds(p, 16, bounds, pt, dw.seq_lens, device(blocks), out)
        idx = torch.empty(2 * n, 8, 8, dtype=torch.int32, device="cuda")
        B.attn_select_blocks(p, sparse, dw.q, bounds, pt, dw.seq_lens, dw.qo_indptr, idx)
        assert B.attn_get_device_error(p) == 0
        got.append((out, idx))
        del bounds
    assert torch.equal(got[0][0].view(torch.int16), got[1][0].view(torch.int16)) and torch.equal(got[0][1], got[1][1])
    del k_far
    torch.cuda.empty_cache()


def test_two_plans_at_once():
    """Two plans' steps on two streams, side by side."""
    from asymmetric_kv_paged_gb300 import binding as B
    sets = []
    for seed, kv, seq, n in ((1, "bf16", [900], [300]), (2, "fp8", [2000, 700], [250, 130])):
        w, dw = sparse_setup(kv, seq, n, 16, 2, 64, seed=seed)
        bounds = device(random_bounds(np.random.default_rng(seed), w, 64))
        lists = P_.select(w, w.q, bounds.cpu().numpy(), 64, 6, 1, 1)
        idx = torch.empty(w.total_q, 2, 6, dtype=torch.int32, device="cuda")
        out = torch.empty(w.total_q, 16, 128, dtype=BF, device="cuda")
        sets.append((w, dw, bounds, lists, attend(w, dw, lists, 64)[0], idx, out, torch.cuda.Stream()))
    torch.cuda.synchronize()
    sparse = B.make_sparse(64, 6)
    for _ in range(8):
        for w, dw, bounds, lists, o, idx, out, stream in sets:
            with torch.cuda.stream(stream):
                B.attn_select_blocks(dw.plan, sparse, dw.q, bounds, dw.page_table, dw.seq_lens, dw.qo_indptr, idx)
                B.attn_run_sparse(dw.plan, sparse, dw.q, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens,
                                  dw.qo_indptr, idx, None, w.softmax_scale, w.k_scale, w.v_scale, out)
    torch.cuda.synchronize()
    for w, dw, bounds, lists, o, idx, out, stream in sets:
        assert np.array_equal(idx.cpu().numpy(), lists)
        assert np.array_equal(out.double().cpu().numpy(), o)
        assert B.attn_get_device_error(dw.plan) == 0


def test_shifts_out_of_every_range_skip_their_tokens():
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = sparse_setup("bf16", [60, 60, 60], [1, 1, 1], 8, 2, 16)
    tab = torch.zeros(64, 64, device="cuda")
    delta = device(np.array([2 ** 31 - 1, -2 ** 31, 3], np.int32))
    mrope = B.make_mrope(tab, 64, B.mrope_axes([8, 12, 12]), position_delta=delta)
    kn, vn = torch.ones(3, 2, 192, dtype=BF, device="cuda"), torch.ones(3, 2, 128, dtype=BF, device="cuda")
    q_out = torch.full_like(dw.q, 7.0)
    B.attn_append_kv_mrope(dw.plan, mrope, dw.q, kn, vn, q_out, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens,
                           dw.qo_indptr)
    assert B.attn_get_device_error(dw.plan) == 8
    assert (q_out == 7).all((1, 2)).tolist() == [True, True, False]


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_rows_beside_nans_of_a_mixed_batch(kv):
    """Decode requests beside a chunk of tokens, sinks, lists in any order, one value of a block NaN:
    the dims of the rows that list it, and the other rows stay close to the 64-bit form; without
    lse_out the same bits."""
    from asymmetric_kv_paged_gb300 import binding as B
    seq, n = [900] * 40 + [700], [1] * 40 + [250]
    w, dw = sparse_setup(kv, seq, n, 16, 2, 64, sinks=True)
    lists = random_lists(np.random.default_rng(3), w, 64, 6)
    lists = np.random.default_rng(4).permuted(lists, axis=-1)
    ref = P_.attend(w, w.q, 64, lists, w.sinks)
    flat = dw.v_cache.view(-1, *dw.v_cache.shape[2:])
    slot = int(P_.slots(w, 40, 3 * 64 + 5))                        # key 197 of the chunk's request, head 1
    if kv == "fp4":
        flat[slot, 1, 64] = 0x7F                                   # the scale of dims 0 to 15
    else:
        flat[slot, 1, 7] = float("nan") if kv == "bf16" else 0x7F
    dims = slice(0, 16) if kv == "fp4" else slice(7, 8)
    o, l = attend(w, dw, lists, 64)
    hit = (lists[:, 1] == 3).any(-1) & (np.arange(w.total_q) >= 40)
    assert 20 < hit.sum() < 240
    assert np.isnan(o[hit, 8:, dims]).all() and not np.isnan(o[~hit]).any() and not np.isnan(o[:, :8]).any()
    rows = np.ones((w.total_q, 16), bool)
    rows[hit, 8:] = False
    P_.assert_close(o[rows], l[rows], [x[rows] for x in ref], kv)
    clean = np.ones(128, bool)
    clean[dims] = False
    tol = [x[hit, 8:][..., clean] if x.ndim == 3 else x[hit, 8:] for x in ref]
    P_.assert_close(o[hit, 8:][..., clean], l[hit, 8:], tol, kv)
    out = torch.empty(w.total_q, 16, 128, dtype=BF, device="cuda")
    B.attn_run_sparse(dw.plan, B.make_sparse(64, 6, 0, 1), dw.q, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens,
                      dw.qo_indptr, device(lists), dw.sinks, w.softmax_scale, w.k_scale, w.v_scale, out)
    assert np.array_equal(out.double().cpu().numpy(), o, equal_nan=True)
    assert B.attn_get_device_error(dw.plan) == 0
