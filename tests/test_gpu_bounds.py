"""attn_update_bounds and attn_read_bounds: records bit for bit against the definition."""
import numpy as np
import pytest

import sparse_plain as P_
from asymmetric_kv_paged_gb300 import workloads as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def setup(kv, seq, n, P, dqk=192, hkv=2, seed=5, **kw):
    from asymmetric_kv_paged_gb300 import binding as B
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    w = W.make_workload(seed, seq, n, hq=2 * hkv, hkv=hkv, page_size=P, kv_dtype=kv, dqk=dqk, **kw)
    return w, DeviceWorkload(w), B.attn_bounds_row_bytes(dqk)


def device(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def indptr(counts):
    return np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)


def update(dw, block, bounds, ind, lens=None, pt=None):
    from asymmetric_kv_paged_gb300 import binding as B
    B.attn_update_bounds(dw.plan, block, dw.k_cache, bounds, dw.page_table if pt is None else pt,
                         dw.seq_lens if lens is None else lens, device(ind), int(ind[-1]))


CASES = [
    # kv, dqk, hkv, P, block, seq_lens, new rows
    ("bf16", 192, 2, 64, 64, [300, 64, 63, 128], [300, 64, 63, 1]),
    ("fp8", 192, 3, 64, 32, [300, 64, 65], [40, 64, 2]),
    ("fp4", 192, 1, 128, 128, [700, 128, 127], [600, 1, 127]),
    ("bf16", 128, 4, 48, 16, [100, 16, 15, 49], [1, 1, 15, 49]),
    ("fp8", 128, 1, 384, 128, [1000], [1000]),
    ("fp4", 128, 2, 32, 16, [500, 33, 32], [500, 2, 0]),
    ("bf16", 192, 2, 64, 64, list(range(60, 130)), [3] * 70),
    ("fp8", 192, 8, 128, 64, [4000, 3000], [4000, 3000]),
]


@pytest.mark.parametrize("kv,dqk,hkv,P,block,seq,new", CASES)
def test_records_of_completed_blocks(kv, dqk, hkv, P, block, seq, new):
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw, row = setup(kv, seq, new, P, dqk, hkv)
    rng = np.random.default_rng(1)
    before = rng.integers(0, 256, (w.num_pages, P // block, hkv, row), dtype=np.uint8)
    bounds = device(before)
    ind = indptr(new)
    update(dw, block, bounds, ind)
    ref = P_.update_bounds(w, before, block, w.k_cache, w.seq_lens, ind)
    assert B.attn_get_device_error(dw.plan) == 0
    assert np.array_equal(bounds.cpu().numpy(), ref)          # other blocks' records as they were
    # read back: the blocks just completed
    seq_, new_ = np.array(seq), np.array(new)
    done = seq_ // block - (seq_ - new_) // block
    bi = indptr(done)
    out = torch.full((int(bi[-1]), hkv, 2, dqk), 7.0, dtype=BF, device="cuda")
    B.attn_read_bounds(dw.plan, block, bounds, dw.page_table, dw.seq_lens, device(bi), out)
    assert B.attn_get_device_error(dw.plan) == 0
    want = []
    flat = ref.reshape(-1, hkv, row).view(np.int8).astype(np.float64)
    for b in range(len(seq)):
        for c in range(seq[b] // block - done[b], seq[b] // block):
            r = flat[int(P_.slots(w, b, c * block)) // block]
            want.append(r[:, :2 * dqk].reshape(hkv, 2, dqk) * 2.0 ** r[:, 2 * dqk][:, None, None])
    if want:
        assert np.array_equal(out.double().cpu().numpy(), np.array(want))


def test_records_bound_every_key_and_extremes():
    """Zeros, subnormals, the largest values, one large value among small ones, NaN, infinities."""
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw, row = setup("bf16", [64 * 9], [1], 64)
    k = w.k_cache.reshape(-1, 2, 192).copy()
    s = [int(P_.slots(w, 0, 64 * c)) for c in range(9)]
    bits = W.bf16_bits
    k[s[0]:s[0] + 64] = 0
    k[s[1]:s[1] + 64] = 0x8000                                    # minus zero
    k[s[2]:s[2] + 64] = np.random.default_rng(1).integers(1, 128, (64, 2, 192))            # subnormals
    k[s[3] + 5, 1, 7] = bits(np.float32([1.984375 * 2.0 ** 20]))[0]                        # 127 * 2^14
    k[s[4] + 63, 0, 191] = bits(np.float32([-1.9921875 * 2.0 ** 20]))[0]                   # above it
    k[s[5], 0, 0] = 0x7FC0
    k[s[6] + 63, 1, 0] = 0x7F80
    k[s[7] + 8, 0, 100] = 0xFF80
    k[s[8] + 1, 1, 3] = 0x7F7F                                                            # the largest bf16
    dw.k_cache.copy_(torch.from_numpy(k.view(np.int16)).view(BF).cuda().view(dw.k_cache.shape))
    bounds = torch.zeros(w.num_pages, 1, 2, row, dtype=torch.uint8, device="cuda")
    ind = indptr([64 * 9])
    update(dw, 64, bounds, ind)
    kc = k.reshape(w.k_cache.shape)
    ref = P_.update_bounds(w, np.zeros(bounds.shape, np.uint8), 64, kc, w.seq_lens, ind)
    assert np.array_equal(bounds.cpu().numpy(), ref)
    out = torch.empty(9, 2, 2, 192, dtype=BF, device="cuda")
    B.attn_read_bounds(dw.plan, 64, bounds, dw.page_table, dw.seq_lens, device(indptr([9])), out)
    v = W.bf16_values(k)
    got = out.float().cpu().numpy()
    with np.errstate(invalid="ignore"):
        for c in range(9):
            for g in range(2):
                rows = v[s[c]:s[c] + 64, g]
                assert np.all((rows <= got[c, g, 0]) | np.isnan(rows)) and np.all((rows >= got[c, g, 1]) | np.isnan(rows))
                if not np.isfinite(rows).all():
                    assert np.all(got[c, g, 0] == np.inf) and np.all(got[c, g, 1] == -np.inf)
    assert B.attn_get_device_error(dw.plan) == 0


@pytest.mark.parametrize("kv", ["fp8", "fp4"])
def test_nan_codes_make_an_odd_block(kv):
    w, dw, row = setup(kv, [128], [128], 64)
    k = w.k_cache.reshape(-1, 2, w.k_cache.shape[-1]).copy()
    s = int(P_.slots(w, 0, 64))
    k[s + 9, 1, 50 if kv == "fp8" else 96 + 3] = 0x7F
    dw.k_cache.copy_(torch.from_numpy(k).cuda().view(dw.k_cache.shape))
    bounds = torch.zeros(w.num_pages, 1, 2, row, dtype=torch.uint8, device="cuda")
    ind = indptr([128])
    update(dw, 64, bounds, ind)
    ref = P_.update_bounds(w, np.zeros(bounds.shape, np.uint8), 64, k.reshape(w.k_cache.shape), w.seq_lens, ind)
    assert ref.reshape(-1, 2, row)[s // 64, 1, 384] == 127
    assert np.array_equal(bounds.cpu().numpy(), ref)


def test_bad_pages_and_lengths_are_skipped():
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw, row = setup("bf16", [128, 128, 128], [64, 64, 64], 64)
    bounds = torch.zeros(w.num_pages, 1, 2, row, dtype=torch.uint8, device="cuda")
    pt = dw.page_table.clone()
    pt[0, 1] = w.num_pages
    ind = indptr([64, 64, 64])
    update(dw, 64, bounds, ind, pt=pt)
    assert B.attn_get_device_error(dw.plan) == 1
    lens = torch.tensor([128, 20, 64 * (dw.page_table.shape[1] + 1)], dtype=torch.int32, device="cuda")
    update(dw, 64, bounds, ind, lens=lens)                       # positions before 0, and past the table's row
    assert B.attn_get_device_error(dw.plan) == 4
    short = np.array([0, 64, 100, 128], np.int32)                 # rows past kv_indptr's last
    B.attn_update_bounds(dw.plan, 64, dw.k_cache, bounds, dw.page_table, dw.seq_lens, device(short), 192)
    assert B.attn_get_device_error(dw.plan) == 4
    out = torch.full((5, 2, 2, 192), 7.0, dtype=BF, device="cuda")
    B.attn_read_bounds(dw.plan, 64, bounds, pt, lens, device(np.array([0, 1, 2, 4], np.int32)), out)
    assert B.attn_get_device_error(dw.plan) == 1 | 4
    # a bad page; a block before 0 of a request of 20; a block past the table and one within; past the last
    zero = (out == 0).all(-1).all(-1).all(-1).cpu().tolist()
    assert zero[0] and zero[1] and zero[3] and zero[4]


def test_refusals():
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw, row = setup("bf16", [100], [4], 48)
    bounds = torch.zeros(w.num_pages, 3, 2, row, dtype=torch.uint8, device="cuda")
    out = torch.empty(2, 2, 2, 192, dtype=BF, device="cuda")
    I, S = B.ATTN_ERR_INVALID_ARG, B.ATTN_ERR_UNSUPPORTED
    base = dict(block=16, k=dw.k_cache, b=bounds, pt=dw.page_table, ind=dw.qo_indptr, rows=4)

    def call(**kw):
        a = {**base, **kw}
        B.attn_update_bounds(dw.plan, a["block"], a["k"], a["b"], a["pt"], dw.seq_lens, a["ind"], a["rows"])

    odd = torch.zeros(bounds.numel() + 8, dtype=torch.uint8, device="cuda")[8:]
    for kw, status in ((dict(block=0), S), (dict(block=24), S), (dict(block=64), S), (dict(block=-16), S),
                       (dict(k=None), I), (dict(b=None), I), (dict(pt=None), I), (dict(ind=None), I),
                       (dict(rows=-1), I), (dict(b=odd), I)):
        with pytest.raises(B.AttnError) as e:
            call(**kw)
        assert e.value.status == status, kw
    for kw, status in ((dict(b=None), I), (dict(ind=None), I), (dict(block=32), S)):
        a = {**base, **kw}
        with pytest.raises(B.AttnError) as e:
            B.attn_read_bounds(dw.plan, a["block"], a["b"], a["pt"], dw.seq_lens, a["ind"], out)
        assert e.value.status == status, kw
    call(rows=0)                                                 # no rows, no work
    torch.cuda.synchronize()
    assert int(bounds.sum()) == 0 and B.attn_get_device_error(dw.plan) == 0
