"""attn_append_kv_mrope: caches and rotated queries bit for bit against fp32 arithmetic with a
table row per (token, pair)."""
import numpy as np
import pytest

from asymmetric_kv_paged_gb300 import workloads as W
from oracle import append as A

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

BF = torch.bfloat16


def table(max_pos, rot):
    inv = 10000.0 ** (-np.arange(rot // 2) / (rot // 2))
    ang = np.arange(max_pos)[:, None] * inv
    return np.concatenate([np.cos(ang), np.sin(ang)], -1).astype(np.float32)


def device(x):
    return torch.from_numpy(np.ascontiguousarray(x)).cuda()


def rows(rng, *shape):
    return W.bf16_bits((rng.standard_normal(shape) * 2).astype(np.float32))


def dev(bits):
    return device(bits.view(np.int16)).view(BF)


def bits(t):
    return t.contiguous().view(torch.int16 if t.dtype == BF else torch.uint8).cpu().numpy().view(
        np.uint16 if t.dtype == BF else np.uint8)


def setup(kv, seq, n, hq, hkv, P, dqk):
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    w = W.make_workload(3, seq, n, hq=hq, hkv=hkv, page_size=P, kv_dtype=kv, dqk=dqk)
    return w, DeviceWorkload(w)


def own_positions(w):
    return np.concatenate([np.arange(L - (b - a), L) for L, a, b in
                           zip(w.seq_lens, w.qo_indptr[:-1], w.qo_indptr[1:])]).astype(np.int64)


CASES = [
    # kv, seq_lens, n, hq, hkv, P, dqk, rot, off, interleaved, pair axes, positions
    ("bf16", [1000, 129, 3000], [1, 1, 1], 16, 2, 128, 192, 64, 0, False, [8, 12, 12], "given"),
    ("fp8", [700, 40], [8, 8], 16, 2, 16, 192, 64, 128, True, [8, 12, 12], "given"),
    ("fp4", [700, 40], [8, 8], 16, 2, 16, 192, 64, 128, True, "turns", "delta"),
    ("fp4", [300], [120], 8, 1, 1, 192, 192, 0, False, "turns", "given"),
    ("bf16", [260], [133], 16, 4, 3, 192, 48, 8, False, "random", "given"),
    ("fp8", [90, 50, 20], [5, 0, 3], 8, 2, 3, 192, 112, 40, False, "random", "delta"),
    ("fp4", [90, 50, 20], [5, 0, 3], 8, 2, 64, 128, 128, 0, True, "random", "given"),
    ("bf16", [90, 33], [1, 33], 15, 3, 8, 128, 80, 48, False, [16, 24], "own"),
    ("bf16", [90, 33], [1, 33], 15, 3, 8, 128, 16, 8, True, "one", "given"),
    ("fp8", [2999, 3000, 7, 1], [2400, 2470, 0, 1], 3, 1, 16, 128, 64, 64, True, "turns", "given"),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("kv,seq,n,hq,hkv,P,dqk,rot,off,inter,axes,where", CASES)
def test_bit_exact(kv, seq, n, hq, hkv, P, dqk, rot, off, inter, axes, where, in_place):
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup(kv, seq, n, hq, hkv, P, dqk)
    rng = np.random.default_rng(7)
    half = rot // 2
    if axes == "turns":
        axes = B.mrope_axes([half - 2 * (half // 3), half // 3, half // 3], in_turn=True)
    elif axes == "random":
        axes = rng.integers(0, 4, half).tolist()
    elif axes == "one":
        axes = [0] * half
    else:
        axes = B.mrope_axes(axes)
    A_ = max(axes) + 1
    kn, vn = rows(rng, w.total_q, hkv, dqk), rows(rng, w.total_q, hkv, 128)
    tab = table(3100, rot)
    kw = {}
    if where == "given":
        pos = rng.integers(0, 3100, (A_, w.total_q))
        kw["positions"] = device(pos.astype(np.int32))
    else:
        pos = np.broadcast_to(own_positions(w), (A_, w.total_q))
        if where == "delta":
            d = np.array([-17, 5, 30][:w.batch], np.int32)
            pos = pos + np.repeat(d, np.diff(w.qo_indptr))
            kw["position_delta"] = device(d)
    at = pos[np.array(axes)].T                                     # [T, half]
    i = np.arange(half)
    cs = np.concatenate([tab[at, i], tab[at, half + i]], -1)[:, None]
    ks, vs = (0.0173, 0.0091) if kv == "fp4" else (w.k_scale, w.v_scale)
    ref_k, ref_v = A.append_rows(A.rotate(W.bf16_values(kn), cs, rot, off, inter), W.bf16_values(vn), w.k_cache,
                                 w.v_cache, w.page_table, w.seq_lens, w.qo_indptr, kv, ks, vs)
    ref_q = A.f32_to_bf16(A.rotate(W.bf16_values(w.q), cs, rot, off, inter))
    mrope = B.make_mrope(device(tab), rot, axes, rot_offset=off, interleaved=inter, **kw)
    q_out = dw.q if in_place else torch.full_like(dw.q, float("nan"))
    B.attn_append_kv_mrope(dw.plan, mrope, dw.q, dev(kn), dev(vn), q_out, dw.k_cache, dw.v_cache, dw.page_table,
                           dw.seq_lens, dw.qo_indptr, ks, vs)
    torch.cuda.synchronize()
    assert B.attn_get_device_error(dw.plan) == 0
    assert np.array_equal(bits(dw.k_cache).reshape(ref_k.shape), ref_k)
    assert np.array_equal(bits(dw.v_cache).reshape(ref_v.shape), ref_v)
    assert np.array_equal(bits(q_out), ref_q)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
def test_equal_positions_are_the_rotation_of_one_axis(kv):
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup(kv, [300, 77], [30, 1], 16, 2, 16, 192)
    rng = np.random.default_rng(7)
    kn, vn = dev(rows(rng, 31, 2, 192)), dev(rows(rng, 31, 2, 128))
    tab = device(table(400, 96))
    k0, v0 = dw.k_cache.clone(), dw.v_cache.clone()
    got = []
    for how in range(2):
        dw.k_cache.copy_(k0), dw.v_cache.copy_(v0)
        q_out = torch.empty_like(dw.q)
        args = (dw.q, kn, vn, q_out, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens, dw.qo_indptr, w.k_scale,
                w.v_scale)
        if how:
            B.attn_append_kv_mrope(dw.plan, B.make_mrope(tab, 96, B.mrope_axes([16, 16, 16])), *args)
        else:
            B.attn_append_kv_rope(dw.plan, B.make_rope(tab, 96), *args)
        got.append([bits(q_out), bits(dw.k_cache), bits(dw.v_cache)])
    assert all(np.array_equal(a, b) for a, b in zip(*got))


def test_positions_outside_the_table_skip_their_token():
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup("bf16", [60], [4], 8, 2, 16, 192)
    rng = np.random.default_rng(2)
    kn, vn = dev(rows(rng, 4, 2, 192)), dev(rows(rng, 4, 2, 128))
    pos = np.array([[1, 2, 3, 4], [1, 58, 3, 4], [1, 2, -1, 4]], np.int32)
    before = bits(dw.k_cache).copy()
    q_out = torch.zeros_like(dw.q)
    mrope = B.make_mrope(device(table(58, 64)), 64, B.mrope_axes([8, 12, 12]), positions=device(pos))
    B.attn_append_kv_mrope(dw.plan, mrope, dw.q, kn, vn, q_out, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens,
                           dw.qo_indptr)
    torch.cuda.synchronize()
    assert B.attn_get_device_error(dw.plan) == 8
    assert (bits(q_out) != 0).any((1, 2)).tolist() == [True, False, False, True]
    changed = (bits(dw.k_cache) != before).reshape(-1, 2 * 192).any(-1)
    at = [int(w.page_table[0, p // 16]) * 16 + p % 16 for p in (56, 59)]
    assert sorted(np.flatnonzero(changed).tolist()) == sorted(at)


def test_refusals():
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup("bf16", [60], [2], 8, 2, 16, 192)
    rng = np.random.default_rng(2)
    kn, vn = dev(rows(rng, 2, 2, 192)), dev(rows(rng, 2, 2, 128))
    tab = device(table(100, 64))
    before = bits(dw.k_cache).copy()

    def call(change=lambda m: None, **kw):
        m = B.make_mrope(tab, 64, B.mrope_axes([8, 12, 12]), **kw)
        change(m)
        B.attn_append_kv_mrope(dw.plan, m, dw.q, kn, vn, dw.q, dw.k_cache, dw.v_cache, dw.page_table, dw.seq_lens,
                               dw.qo_indptr)

    def no_axes(m): m.num_axes = 0
    def many(m): m.num_axes = 5
    def fewer(m): m.num_axes = 2
    def null(m): m.pair_axis_host = None
    def odd(m): m.rope.rot_dim = 24
    def far(m): m.rope.rot_offset = 136
    def empty(m): m.rope.max_pos = 0
    both = dict(positions=torch.zeros(3, 2, dtype=torch.int32, device="cuda"),
                position_delta=torch.zeros(1, dtype=torch.int32, device="cuda"))
    I, S = B.ATTN_ERR_INVALID_ARG, B.ATTN_ERR_UNSUPPORTED
    for change, status in ((no_axes, I), (many, I), (fewer, I), (null, I), (odd, S), (far, I), (empty, I)):
        with pytest.raises(B.AttnError) as e:
            call(change)
        assert e.value.status == status, change.__name__
    with pytest.raises(B.AttnError) as e:
        call(**both)
    assert e.value.status == I
    torch.cuda.synchronize()
    assert np.array_equal(bits(dw.k_cache), before) and B.attn_get_device_error(dw.plan) == 0
