"""The rotating append and the reading back where a warp takes many rows of a token:
chunks of over a thousand tokens of many heads, bit for bit, in place and not."""
import numpy as np
import pytest

from asymmetric_kv_paged_gb300 import workloads as W
from oracle import append as A

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_rope import bits, dev, positions, rows, same_caches, setup, table  # noqa: E402


def stored(x, kv, scale):
    """What a cache holds of fp32 rows (array forms of the oracle's encoders: the host
    tests hold the two equal)."""
    if kv == "bf16":
        return A.f32_to_bf16(x)
    y = (x / np.float32(scale)).astype(np.float32)
    if kv == "fp8":
        return W.e4m3_codes(np.clip(y, -448, 448))
    return W.fp4_rows(y)


CASES = [
    # kv, seq_lens, n, hq, hkv, P, dqk, rot, off, interleaved, given positions
    ("fp8", [1500], [1300], 64, 8, 16, 192, 64, 0, False, False),
    ("fp4", [1500, 40], [1300, 3], 64, 8, 16, 192, 64, 128, True, False),
    ("bf16", [700, 900], [650, 655], 64, 8, 1, 192, 192, 0, False, True),
    ("fp4", [1300], [1300], 40, 20, 128, 128, 48, 80, False, True),
    ("fp8", [2600, 2500], [2450, 2450], 33, 11, 3, 128, 128, 0, True, False),
    ("bf16", [5000], [4900], 24, 12, 16, 128, 64, 64, False, False),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}_{sum(c[2])}x{c[3]}x{c[4]}")
def test_many_rows_of_a_token(case, in_place):
    from asymmetric_kv_paged_gb300 import binding as B
    kv, seq, n, hq, hkv, P, dqk, rot, off, inter, given = case
    w, dw = setup(kv, seq, n, hq, hkv, P, dqk)
    rng = np.random.default_rng(17)
    kn, vn = rows(rng, w.total_q, hkv, dqk), rows(rng, w.total_q, hkv, 128)
    tab = table(5000, rot)
    pos = rng.integers(0, 5000, w.total_q) if given else positions(w)
    ks, vs = (0.0173, 0.0091) if kv == "fp4" else (w.k_scale, w.v_scale)
    cs = tab[pos][:, None]
    own = positions(w)
    req = np.repeat(np.arange(w.batch), np.diff(w.qo_indptr))
    slot = w.page_table[req, own // P].astype(np.int64) * P + own % P
    ref_k, ref_v = w.k_cache.copy(), w.v_cache.copy()
    for ref, x, sc in ((ref_k, A.rotate(W.bf16_values(kn), cs, rot, off, inter), ks), (ref_v, W.bf16_values(vn), vs)):
        ref.reshape((-1,) + ref.shape[2:])[slot] = stored(x, kv, sc)
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
    if not in_place:
        assert np.array_equal(bits(dw.q), w.q)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("hkv,dqk", [(12, 192), (20, 128)])
def test_reading_many_rows_of_many_heads(kv, hkv, dqk):
    from asymmetric_kv_paged_gb300 import binding as B
    P = 16
    w, dw = setup(kv, [3000, 1999], [1, 1], hq=hkv, hkv=hkv, P=P, dqk=dqk)
    ks, vs = (1.0, 1.0) if kv == "bf16" else (w.k_scale, 0.37)
    ind = np.array([0, 3000, 4999], np.int32)
    ko = torch.full((4999, hkv, dqk), 7.0, dtype=torch.bfloat16, device="cuda")
    vo = torch.full((4999, hkv, 128), 7.0, dtype=torch.bfloat16, device="cuda")
    B.attn_read_kv(dw.plan, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens, torch.from_numpy(ind).cuda(), ko, vo,
                   ks, vs)
    pos = np.concatenate([np.arange(3000), np.arange(1999)])
    slot = w.page_table[np.repeat([0, 1], [3000, 1999]), pos // P].astype(np.int64) * P + pos % P
    for cache, out, d, sc in ((w.k_cache, ko, dqk, ks), (w.v_cache, vo, 128, vs)):
        r = cache.reshape(-1, hkv, cache.shape[-1])[slot]
        if kv == "bf16":
            want = r
        elif kv == "fp8":
            want = A.f32_to_bf16(torch.from_numpy(r.copy()).view(torch.float8_e4m3fn).float().numpy() * np.float32(sc))
        else:
            want = A.f32_to_bf16(W.fp4_values(r, d) * np.float32(sc))
        assert np.array_equal(bits(out), want)
    assert B.attn_get_device_error(dw.plan) == 0
