"""attn_select_blocks: the lists equal the definition's, ties and extremes included."""
import numpy as np
import pytest

import sparse_plain as P_
from asymmetric_kv_paged_gb300 import workloads as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def setup(seq, n, hq, hkv, P, dqk=192, seed=5, replayable=False):
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    w = W.make_workload(seed, seq, n, hq=hq, hkv=hkv, page_size=P, kv_dtype="bf16", dqk=dqk)
    return w, DeviceWorkload(w, replayable=replayable)


def random_bounds(rng, w, block, spread=40):
    """Records of every kind of magnitude: upper and lower codes, and exponents that differ."""
    from asymmetric_kv_paged_gb300 import binding as B
    rec = np.zeros((w.num_pages, w.page_size // block, w.hkv, B.attn_bounds_row_bytes(w.dqk)), np.int8)
    mid = rng.integers(-60, 61, rec.shape[:-1] + (w.dqk,))
    r = rng.integers(0, spread, rec.shape[:-1] + (w.dqk,))
    rec[..., :w.dqk], rec[..., w.dqk:2 * w.dqk] = mid + r, mid - r
    rec[..., 2 * w.dqk] = rng.integers(-6, -3, rec.shape[:-1])
    return rec.view(np.uint8)


def device(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def run(w, dw, q, bounds, block, take, first, last, seq_lens=None, pt=None):
    from asymmetric_kv_paged_gb300 import binding as B
    out = torch.full((w.total_q + 1, w.hkv, take), -7, dtype=torch.int32, device="cuda")
    B.attn_select_blocks(dw.plan, B.make_sparse(block, take, first, last), device(q.view(np.int16)).view(BF),
                         device(bounds), dw.page_table if pt is None else pt,
                         dw.seq_lens if seq_lens is None else seq_lens, dw.qo_indptr, out[:w.total_q])
    out = out.cpu().numpy()
    assert (out[w.total_q] == -7).all()                          # behind the last token: as it was
    return out[:w.total_q]


CASES = [
    # seq_lens, n, hq, hkv, P, dqk, block, take, first, last
    ([3000, 700, 64, 1, 1025], [1] * 5, 16, 2, 64, 192, 64, 16, 1, 2),
    ([3000, 700, 64, 1, 1025], [1] * 5, 8, 1, 16, 128, 16, 40, 0, 1),
    ([2000, 300], [8, 3], 64, 4, 128, 192, 32, 8, 2, 3),
    ([900], [333], 12, 3, 64, 192, 16, 7, 1, 1),
    ([700, 20, 5], [130, 20, 0], 40, 2, 128, 128, 64, 4, 0, 2),
    ([600, 500], [1, 60], 4, 4, 32, 192, 32, 5, 1, 1),
    ([9000], [1], 128, 1, 128, 192, 128, 3, 1, 1),               # eight row tiles
    ([5000], [2], 21, 1, 48, 192, 16, 256, 3, 2),                 # two row tiles, the longest list
    ([257] * 40, [1] * 40, 8, 2, 64, 192, 64, 2, 1, 1),           # nothing but forced blocks
    ([40000], [1], 16, 2, 64, 192, 16, 64, 1, 1),                 # 2,500 blocks
    ([40000], [2], 16, 1, 64, 128, 16, 3, 2, 1),                  # nothing but forced blocks of many
    ([9000, 30000], [1, 1], 8, 1, 32, 192, 16, 17, 0, 2),         # 562 and 1,875
    ([1000] * 300, [1] * 300, 16, 1, 64, 128, 64, 6, 1, 2),       # one CTA a token
    ([1500, 31, 800], [200, 31, 77], 16, 1, 32, 192, 32, 12, 1, 2),
    ([1100], [530], 32, 2, 16, 128, 16, 20, 0, 3),
    # chunks of tokens: token tiles of 8, 4, 2, 1, 32, 128 tokens; lists that take all; several block tiles
    ([5000], [700], 16, 1, 64, 192, 16, 30, 2, 2),
    ([900, 700, 64, 1], [300, 411, 64, 1], 64, 2, 32, 192, 16, 9, 1, 1),
    ([700], [333], 50, 1, 16, 128, 16, 9, 0, 1),
    ([600], [333], 96, 1, 16, 192, 16, 9, 1, 2),
    ([2100], [500], 12, 3, 48, 128, 16, 11, 1, 1),
    ([600, 2500], [150, 600], 3, 3, 64, 192, 16, 25, 1, 3),
    ([400], [390], 16, 2, 64, 192, 64, 7, 1, 1),
]


@pytest.mark.parametrize("seq,n,hq,hkv,P,dqk,block,take,first,last", CASES)
def test_lists(seq, n, hq, hkv, P, dqk, block, take, first, last):
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup(seq, n, hq, hkv, P, dqk)
    bounds = random_bounds(np.random.default_rng(3), w, block)
    got = run(w, dw, w.q, bounds, block, take, first, last)
    assert B.attn_get_device_error(dw.plan) == 0
    assert np.array_equal(got, P_.select(w, w.q, bounds, block, take, first, last))


@pytest.mark.parametrize("n", [2, 400])
def test_scores_are_exact_at_the_codes_ends(n):
    """Every product at its largest: 192 * 127 * 127 in magnitude, apart by single units."""
    w, dw = setup([4000], [n], 16, 1, 64)
    rng = np.random.default_rng(1)
    bounds = random_bounds(rng, w, 64).view(np.int8)
    bounds[..., :384] = rng.choice([-127, 126, 127], bounds.shape[:-1] + (384,))
    bounds[..., 192:384] = np.minimum(bounds[..., :192], bounds[..., 192:384])
    bounds[..., 384] = 0
    q = W.bf16_bits(np.where(rng.random((n, 16, 192)) < 0.5, -127.0, 127.0).astype(np.float32))
    got = run(w, dw, q, bounds.view(np.uint8), 64, 9, 1, 1)
    assert np.array_equal(got, P_.select(w, q, bounds.view(np.uint8), 64, 9, 1, 1))


@pytest.mark.parametrize("n", [1, 200])
def test_ties_take_the_lowest_index(n):
    w, dw = setup([4096, 4096], [n, 3 * n], 16, 2, 64)
    bounds = random_bounds(np.random.default_rng(1), w, 64, spread=2)
    bounds[...] = bounds[:1]                                      # every block alike
    got = run(w, dw, w.q, bounds, 64, 10, 1, 2)
    assert np.array_equal(got, P_.select(w, w.q, bounds, 64, 10, 1, 2))
    assert got[-1, 0].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 62, 63]
    w2, dw2 = setup([20000], [1], 16, 2, 16)                      # more than a warp holds
    alike = random_bounds(np.random.default_rng(1), w2, 16, spread=2)
    alike[...] = alike[:1]
    got = run(w2, dw2, w2.q, alike, 16, 10, 1, 2)
    assert got[0, 1].tolist() == [0, 1, 2, 3, 4, 5, 6, 7, 1248, 1249]
    few = bounds.view(np.int8).copy()                             # two values only, heads of zeros too
    few[::3, ..., 384] += 1
    q = w.q.copy()
    q[0, :8] = 0
    assert np.array_equal(run(w, dw, q, few.view(np.uint8), 64, 10, 1, 2),
                          P_.select(w, q, few.view(np.uint8), 64, 10, 1, 2))


@pytest.mark.parametrize("n", [1, 120])
def test_odd_blocks_and_odd_queries(n):
    w, dw = setup([3000, 3000], [2 * n, n], 16, 2, 64)
    rng = np.random.default_rng(9)
    bounds = random_bounds(rng, w, 64).view(np.int8)
    for page in rng.choice(w.num_pages, w.num_pages // 4, replace=False):
        bounds[page, 0, rng.integers(2)] = 0
        bounds[page, 0, rng.integers(2), 384] = 127              # holds a NaN: first of all
    q = w.q.copy()
    q[0, 3, 17] = 0x7FC0                                          # a head that takes no part
    q[1, 8:16, 5] = 0x7F80                                        # a whole group
    q[2, 2] = W.bf16_bits(np.full(192, 3e38, np.float32))         # scales far apart
    q[2, 9] = 0x0001
    b = bounds.view(np.uint8)
    for take in (6, 20):
        assert np.array_equal(run(w, dw, q, b, 64, take, 1, 2), P_.select(w, q, b, 64, take, 1, 2))


def test_lengths_are_read_on_the_device_and_clamped():
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup([2000, 900, 400], [1, 4, 1], 16, 2, 64, replayable=True)
    bounds = random_bounds(np.random.default_rng(3), w, 64)
    lens = np.array([1300, 700, 1], np.int32)
    assert np.array_equal(run(w, dw, w.q, bounds, 64, 7, 1, 1, device(lens)),
                          P_.select(w, w.q, bounds, 64, 7, 1, 1, lens))
    assert B.attn_get_device_error(dw.plan) == 0
    # below the new tokens, and past the longest request
    got = run(w, dw, w.q, bounds, 64, 7, 1, 1, device(np.array([5000, 2, -9], np.int32)))
    assert B.attn_get_device_error(dw.plan) == 4
    assert np.array_equal(got, P_.select(w, w.q, bounds, 64, 7, 1, 1, np.array([2000, 4, 1], np.int32)))


def test_pages_outside_the_pool_score_as_zeros():
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup([2000], [1], 16, 2, 64)
    bounds = random_bounds(np.random.default_rng(3), w, 64)
    pt = dw.page_table.clone()
    pt[0, 5], pt[0, 11] = -1, w.num_pages
    got = run(w, dw, w.q, bounds, 64, 7, 1, 1, pt=pt)
    assert B.attn_get_device_error(dw.plan) == 1
    zeros = bounds.copy()
    zeros[w.page_table[0, 5]] = zeros[w.page_table[0, 11]] = 0
    assert np.array_equal(got, P_.select(w, w.q, zeros, 64, 7, 1, 1))


def test_refusals():
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup([300], [2], 16, 2, 64)
    bounds = device(random_bounds(np.random.default_rng(3), w, 64))
    out = torch.full((2, 2, 8), -7, dtype=torch.int32, device="cuda")
    I, S = B.ATTN_ERR_INVALID_ARG, B.ATTN_ERR_UNSUPPORTED

    def call(block=64, take=8, first=1, last=1, q=dw.q, b=bounds, pt=dw.page_table, o=out, plan=dw.plan):
        if o is out and 0 < take <= 4096:
            o = torch.full((2, 2, take), -7, dtype=torch.int32, device="cuda")
        B.attn_select_blocks(plan, B.make_sparse(block, take, first, last), q, b, pt, dw.seq_lens, dw.qo_indptr, o)

    for kw, status in ((dict(block=48), S), (dict(block=128), S), (dict(take=257), I), (dict(last=0), I),
                       (dict(first=-1), I), (dict(first=7, last=2), I), (dict(q=None), I), (dict(b=None), I),
                       (dict(pt=None), I),
                       (dict(q=torch.empty(2 * 16 * 192 + 8, dtype=BF, device="cuda")[4:]), I)):
        with pytest.raises(B.AttnError) as e:
            call(**kw)
        assert e.value.status == status, kw
    with pytest.raises(ValueError):                               # a list array of another size
        call(o=out[:1])
    ww = W.make_workload(5, [300], [2], hq=16, hkv=2, page_size=64, kv_dtype="bf16", window=100)
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    with pytest.raises(B.AttnError) as e:
        call(plan=DeviceWorkload(ww).plan)
    assert e.value.status == I
    torch.cuda.synchronize()
    assert (out == -7).all() and B.attn_get_device_error(dw.plan) == 0
