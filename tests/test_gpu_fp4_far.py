"""4-bit pools whose rows lie more than 2^32 bytes in: attention on every kernel and
page kind, the rotating append and the reading back, at the pool's end, equal bit for
bit to the same pages in a small pool."""
import numpy as np
import pytest

from asymmetric_kv_paged_gb300 import workloads as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_rope import dev, rows, table  # noqa: E402


@pytest.fixture(scope="module")
def pool():
    """Raw bytes for a K and a V pool, V's over 2^32."""
    n = (1 << 32) + (1 << 24)
    yield torch.empty(n * 7 // 5, dtype=torch.uint8, device="cuda"), torch.empty(n, dtype=torch.uint8, device="cuda")
    torch.cuda.empty_cache()


def far(dw, w, pool):
    """The workload's pages at the end of a pool of whole pages: caches, page table, pages."""
    k, v = dw.k_cache, dw.v_cache
    pages = min(pool[0].numel() // (k[0].numel()), pool[1].numel() // v[0].numel())
    out = []
    for t, raw in ((k, pool[0]), (v, pool[1])):
        big = raw[:pages * t[0].numel()].view(pages, *t.shape[1:])
        big[pages - w.num_pages:] = t
        out.append(big)
    assert (pages - w.num_pages) * v[0].numel() > 1 << 32
    return out[0], out[1], dw.page_table + (pages - w.num_pages), pages


@pytest.mark.parametrize("n,hq,P,dqk", [(1, 16, 128, 192), (2, 16, 1, 192), (8, 16, 16, 192), (8, 16, 3, 128),
                                        (16, 16, 1, 192), (200, 16, 16, 192), (200, 16, 1, 192)])
@pytest.mark.parametrize("replayable", [False, True])
def test_attention_far_into_a_pool(pool, n, hq, P, dqk, replayable):
    from asymmetric_kv_paged_gb300 import binding as B
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    w = W.make_workload(51, [700 + n, n], [n, n], hq=hq, hkv=2, page_size=P, kv_dtype="fp4", dqk=dqk)
    # a NaN scale at the causal edge: found again far into the pool too
    key = 700 + n // 2
    w.v_cache.reshape(-1, 2, 80)[int(w.page_table[0, key // P]) * P + key % P, 1, 66] = 0x7F
    dw = DeviceWorkload(w, replayable=replayable)
    dw.run()
    torch.cuda.synchronize()
    ref, ref_lse = dw.out.clone(), dw.lse.clone()
    kc, vc, pt, pages = far(dw, w, pool)
    prob, keep = dw.problem()
    prob.num_pages = pages
    plan = (B.attn_plan_replayable if replayable else B.attn_plan)(prob, 0, keep)
    dw.out.fill_(float("nan"))
    B.attn_run_paged(plan, dw.q, kc, vc, pt, dw.seq_lens, dw.qo_indptr, None, 0, w.softmax_scale, w.k_scale, w.v_scale,
                     dw.out, dw.lse, torch.empty(max(1, plan.workspace_bytes), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    assert B.attn_get_device_error(plan) == 0
    assert torch.equal(dw.out.view(torch.int16), ref.view(torch.int16)) and torch.equal(dw.lse, ref_lse)


@pytest.mark.parametrize("P,dqk", [(16, 192), (1, 128)])
def test_append_and_read_far_into_a_pool(pool, P, dqk):
    from asymmetric_kv_paged_gb300 import binding as B
    from asymmetric_kv_paged_gb300.runner import DeviceWorkload
    w = W.make_workload(52, [300, 40], [130, 1], hq=8, hkv=2, page_size=P, kv_dtype="fp4", dqk=dqk)
    dw = DeviceWorkload(w)
    rng = np.random.default_rng(3)
    kn, vn = dev(rows(rng, 131, 2, dqk)), dev(rows(rng, 131, 2, 128))
    rope = B.make_rope(torch.from_numpy(table(400, 64)).cuda(), 64)
    kc, vc, pt, pages = far(dw, w, pool)
    prob, keep = dw.problem()
    prob.num_pages = pages
    plan = B.attn_plan(prob, 0, keep)
    got = []
    for p, k, v, t in ((dw.plan, dw.k_cache, dw.v_cache, dw.page_table), (plan, kc, vc, pt)):
        q = torch.empty_like(dw.q)
        B.attn_append_kv_rope(p, rope, dw.q, kn, vn, q, k, v, t, dw.seq_lens, dw.qo_indptr, w.k_scale, w.v_scale)
        ko = torch.empty(131, 2, dqk, dtype=torch.bfloat16, device="cuda")
        vo = torch.empty(131, 2, 128, dtype=torch.bfloat16, device="cuda")
        B.attn_read_kv(p, k, v, t, dw.seq_lens, dw.qo_indptr, ko, vo, w.k_scale, w.v_scale)
        torch.cuda.synchronize()
        assert B.attn_get_device_error(p) == 0
        got.append((q, ko, vo))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    assert torch.equal(kc[pages - w.num_pages:], dw.k_cache) and torch.equal(vc[pages - w.num_pages:], dw.v_cache)
