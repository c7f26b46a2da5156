"""attn_run_sparse: a visible NaN whose key's neighbours weigh nothing still reaches its row.

Keys of one stretch score 0, all others a few hundred: where a row's results of several warps,
CTAs or chains of tiles meet, the stretch's share is 2^-300 or less of the row's, 0 in fp32.  A NaN
in it is still the row's (a NaN score makes the whole row NaN, a NaN in a V row its dims)."""
import numpy as np
import pytest

import sparse_plain as P_
from asymmetric_kv_paged_gb300 import workloads as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_sparse import run  # noqa: E402


def row(kv, d, what):
    """A cached row whose values are all the type's largest (bf16: 4), or zeros; `nan`: zeros
    but for a NaN among dims 0 to 15."""
    if kv == "bf16":
        r = np.full(d, 0x4080 if what == "large" else 0, np.uint16)
        if what == "nan":
            r[5] = 0x7FC0
        return r
    r = np.zeros(d if kv == "fp8" else W.fp4_row_bytes(d), np.uint8)
    if kv == "fp8":
        r[:] = 0x7E if what == "large" else 0
        if what == "nan":
            r[5] = 0x7F
        return r
    if what == "large":
        r[:d // 2], r[d // 2:d // 2 + d // 16] = 0x77, 0x7E
    elif what == "nan":
        r[d // 2] = 0x7F                                          # the scale of dims 0 to 15
    return r


def build(kv, L, n, stretch, nan_at, cache, dqk):
    """Keys of `stretch` score 0, the others a few hundred; NaNs at `nan_at` of head 1, in K or V."""
    w = W.make_workload(5, [L], [n], hq=16, hkv=2, page_size=64, kv_dtype=kv, dqk=dqk)
    w.q[:] = W.bf16_bits(np.float32([4.0]))[0]
    s = P_.slots(w, 0, np.arange(L))
    k, v = w.k_cache.reshape(-1, 2, w.k_cache.shape[-1]), w.v_cache.reshape(-1, 2, w.v_cache.shape[-1])
    k[s] = row(kv, dqk, "large")
    k[s[stretch]] = row(kv, dqk, "zero")
    clean = w.k_cache.copy(), w.v_cache.copy()
    if cache == "k":
        k[s[nan_at], 1] = row(kv, dqk, "nan")
    else:
        v[s[nan_at], 1] = row(kv, 128, "nan")
    return w, clean


def check(w, kv, lists, clean, cache):
    from asymmetric_kv_paged_gb300 import binding as B
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    dw = DeviceWorkload(w)
    o, l = run(w, dw, lists, 64)
    assert B.attn_get_device_error(dw.plan) == 0
    ref = P_.attend(w, w.q, 64, lists, k_cache=clean[0], v_cache=clean[1])
    assert ref[1].min() > 104                                      # nats: 150 in base 2
    P_.assert_close(o[:, :8], l[:, :8], [x[:, :8] for x in ref], kv)
    if cache == "k":
        assert np.isnan(o[:, 8:]).all() and np.isnan(l[:, 8:]).all()
        return
    dims = np.zeros(128, bool)
    dims[slice(0, 16) if kv == "fp4" else slice(5, 6)] = True
    assert np.isnan(o[:, 8:, dims]).all()
    rest = [x[:, 8:][..., ~dims] if x.ndim == 3 else x[:, 8:] for x in ref]
    P_.assert_close(o[:, 8:][..., ~dims], l[:, 8:], rest, kv)


@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("cache", ["k", "v"])
@pytest.mark.parametrize("take,half,whole", [(3, 0, False), (3, 5, True), (3, 2, False), (32, 9, False), (32, 63, True)])
def test_decode(kv, cache, take, half, whole):
    """A warp's 32 keys score 0, one of them NaN or all: one CTA, and a cluster."""
    stretch = np.arange(32 * half, 32 * half + 32)
    w, clean = build(kv, 64 * take, 1, stretch, stretch if whole else stretch[13:14], cache, 192)
    check(w, kv, np.broadcast_to(np.arange(take, dtype=np.int32), (1, 2, take)).copy(), clean, cache)

@pytest.mark.parametrize("kv", ["bf16", "fp8", "fp4"])
@pytest.mark.parametrize("cache", ["k", "v"])
@pytest.mark.parametrize("tiles", [(1,), (0, 2)])
def test_chunk(kv, cache, tiles):
    """Tiles of two blocks, every second one a chain's: one chain's keys score 0, one of them NaN."""
    n, take = 300, 6
    stretch = np.concatenate([np.arange(128 * t, 128 * t + 128) for t in tiles])
    w, clean = build(kv, 64 * take + n, n, stretch, stretch[77:78], cache, 192 if kv != "fp8" else 128)
    check(w, kv, np.broadcast_to(np.arange(take, dtype=np.int32), (n, 2, take)).copy(), clean, cache)
