"""The 4-bit cache format and the rotating append on the CPU: the oracle's codes
against the format and against the workloads' own encoder, the oracle's rotation
against complex arithmetic, and what the library says without a GPU."""
import ctypes

import numpy as np
import pytest

from asymmetric_kv_paged_gb300 import binding as B
from asymmetric_kv_paged_gb300 import workloads as W
from oracle import append as A


def test_e2m1_codes_are_the_nearest_values_with_ties_to_even():
    values = [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    for c, v in enumerate(values):
        assert A.e2m1_encode(v) == c and A.e2m1_encode(-v if v else -0.0) == c | 8
    ties = {0.25: 0, 0.75: 2, 1.25: 2, 1.75: 4, 2.5: 4, 3.5: 6, 5.0: 6, 1e30: 7}
    for x, c in ties.items():
        assert A.e2m1_encode(x) == c and A.e2m1_encode(-x) == c | 8


@pytest.mark.parametrize("d", [128, 192])
def test_two_encoders_and_two_decoders_agree(d):
    rng = np.random.default_rng(d)
    x = (rng.standard_normal((12, d)) * np.exp(rng.uniform(-12, 8, (12, 1)))).astype(np.float32)
    x[0] = 0                                     # a zero scale
    x[1, :16] = 1e30                             # saturates the block scale
    x[2, 16:32] = np.repeat([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], 2)   # ties under scale 1
    x[3] = 1e-4 * np.sign(x[3])                  # below half the smallest scale: codes keep the sign
    rows = W.fp4_rows(x)
    for r in range(len(x)):
        assert np.array_equal(rows[r], A.fp4_row(x[r], 1.0)), r
        assert np.array_equal(W.fp4_values(rows[r], d), A.fp4_row_values(rows[r], d))
    assert rows.shape[-1] == W.fp4_row_bytes(d) == B.attn_kv_row_bytes(B.ATTN_KV_FP4_E2M1, d)
    # what a code stands for: under the top code the value is within half of the
    # widest gap, 1 * scale, and scale <= (max / 6)(1 + 2^-4) + 2^-10 (half a step of
    # a normal, a subnormal E4M3); above it, within max - 6 * scale, where
    # scale >= (max / 6)(1 - 2^-4) - 2^-10 unless it saturates at 448
    blk = np.abs(x[5:]).reshape(-1, d // 16, 16)
    err = np.abs(W.fp4_values(rows[5:], d).reshape(blk.shape) - x[5:].reshape(blk.shape))
    top = blk.max(-1, keepdims=True)
    assert np.all(err <= top * (1 / 6 + 2.0 ** -4) + 6 * 2.0 ** -10 + np.maximum(top - W.FP4_TOP, 0))


def test_bf16_holds_every_code_times_scale():
    scales = np.array([s for s in range(256) if s & 0x7F != 0x7F], np.uint8)
    rows = np.zeros((len(scales), W.fp4_row_bytes(128)), np.uint8)
    rows[:, :64] = np.tile((np.arange(8) * 2 | (np.arange(8) * 2 + 1) << 4).astype(np.uint8), 8)
    rows[:, 64:72] = scales[:, None]
    v = W.fp4_values(rows, 128)
    assert np.array_equal(W.bf16_values(W.bf16_bits(v)), v)
    assert np.array_equal(v.astype(np.float16).astype(np.float32), v)


@pytest.mark.parametrize("interleaved", [False, True])
def test_oracle_rotation_is_a_complex_product(interleaved):
    rng = np.random.default_rng(3)
    x = rng.standard_normal((5, 192)).astype(np.float32)
    ang = rng.uniform(-9, 9, (5, 32))
    got = A.rotate(x, np.concatenate([np.cos(ang), np.sin(ang)], -1), 64, 24, interleaved)
    p = x[:, 24:88].astype(np.float64)
    z = p[:, 0::2] + 1j * p[:, 1::2] if interleaved else p[:, :32] + 1j * p[:, 32:]
    z = z * np.exp(1j * ang)
    want = x.astype(np.float64)
    if interleaved:
        want[:, 24:88:2], want[:, 25:88:2] = z.real, z.imag
    else:
        want[:, 24:56], want[:, 56:88] = z.real, z.imag
    assert np.array_equal(got[:, :24], x[:, :24]) and np.array_equal(got[:, 88:], x[:, 88:])
    # two products and a sum of fp32, and the table's rounding: 4 half steps of |x1| + |x2|
    assert np.abs(got - want).max() <= 4 * 2.0 ** -24 * 2 * np.abs(x).max()


def test_row_bytes():
    for kv, want in ((B.ATTN_KV_BF16, (384, 256)), (B.ATTN_KV_FP8_E4M3, (192, 128)),
                     (B.ATTN_KV_FP4_E2M1, (112, 80))):
        assert tuple(B.attn_kv_row_bytes(kv, d) for d in (192, 128)) == want
    for kv, d in ((3, 192), (B.ATTN_KV_FP4_E2M1, 64), (-1, 128)):
        with pytest.raises(B.AttnError) as e:
            B.attn_kv_row_bytes(kv, d)
        assert e.value.status == B.ATTN_ERR_UNSUPPORTED
    assert B.load().attn_kv_row_bytes(0, 192, None) == B.ATTN_ERR_INVALID_ARG


@pytest.mark.parametrize("hkv", [1, 2, 3, 8, 40])
@pytest.mark.parametrize("num_sms", [1, 7, 152])
def test_fp4_plans_cover_every_key_once_with_the_heads_in_lockstep(hkv, num_sms):
    """The schedule invariants of every plan, static and replayable; where the heads
    divide the CTAs well, CTA c works on head c % heads, on the same tiles as its
    neighbours."""
    from test_abi_host import _check_plan
    for seq, n in (([4000, 900, 77], [1, 8, 1]), ([37], [1]), ([700, 5, 900, 64], [1, 0, 1, 1])):
        w = W.make_workload(0, seq, n, hq=2 * hkv, hkv=hkv, page_size=16, pages_in_order=True)
        prob, keep = B.make_problem(
            batch=w.batch, num_q_heads=w.hq, num_kv_heads=hkv, page_size=16, num_pages=w.num_pages,
            page_table_stride=w.page_table.shape[1], kv_dtype=B.ATTN_KV_FP4_E2M1, window=0,
            has_sinks=False, qo_indptr=w.qo_indptr, seq_lens=w.seq_lens)
        together = hkv > 1 and hkv <= num_sms and 8 * (num_sms % hkv) <= num_sms
        for replayable in (False, True):
            plan = (B.attn_plan_replayable_host if replayable else B.attn_plan_host)(prob, num_sms, keep)
            for lens in ([w.seq_lens, np.maximum(w.seq_lens // 3, n)] if replayable else [w.seq_lens]):
                w2 = W.Workload(**{**w.__dict__, "seq_lens": np.asarray(lens, np.int32)})
                if replayable:
                    assert B.attn_plan_replan_host(plan, lens) == 0
                info = _check_plan(plan, w2, num_sms, replayable=True)   # its balance bound is below
                segs = B.attn_plan_segments(plan)
                loads = np.bincount(segs[:, 0], weights=segs[:, 3] - segs[:, 2], minlength=info["ctas"])
                # shares of eight tiles at least (a unit for each warp), and blocks of up
                # to sixteen whole
                assert loads.max() <= max(16, np.ceil(loads.sum() / (loads > 0).sum()) * 1.25 + 2 + 4 * replayable)
                if not together:
                    continue
                segs, blocks = B.attn_plan_segments(plan), B.attn_plan_blocks(plan)
                work = {}
                for cta, blk, t0, t1, split in segs.tolist():
                    b, g, row0 = blocks[blk][:3].tolist()
                    assert g == cta % hkv
                    work.setdefault(cta, []).append((b, row0, t0, t1, split))
                assert info["ctas"] % hkv == 0
                for c in range(info["ctas"]):
                    assert work.get(c) == work.get(c - c % hkv)


def test_host_plans_and_null_arguments_are_refused():
    prob, keep = B.make_problem(batch=1, num_q_heads=8, num_kv_heads=1, page_size=16, num_pages=9,
                                page_table_stride=4, kv_dtype=B.ATTN_KV_FP4_E2M1, window=0,
                                has_sinks=False, qo_indptr=[0, 1], seq_lens=[20])
    plan = B.attn_plan_host(prob, 152, keep)
    L = B.load()
    rope = B.attn_rope_t(64, None, 100, 64, 0, 0)
    one = [64] * 9
    for p in (plan.handle, None):               # a plan without a device, no plan
        assert L.attn_append_kv_rope(p, ctypes.byref(rope), *one, 1.0, 1.0, None) == B.ATTN_ERR_INVALID_ARG
        assert L.attn_read_kv(p, 64, 64, 64, 64, 64, 1, 64, 64, 1.0, 1.0, None) == B.ATTN_ERR_INVALID_ARG
        assert L.attn_append_kv(p, *[64] * 7, 1.0, 1.0, None) == B.ATTN_ERR_INVALID_ARG
    assert L.attn_append_kv_rope(plan.handle, None, *one, 1.0, 1.0, None) == B.ATTN_ERR_INVALID_ARG


def test_make_rope_checks_what_the_library_cannot_see():
    torch = pytest.importorskip("torch")
    tab = torch.zeros(10, 64)
    assert (lambda r: (r.max_pos, r.rot_dim, r.rot_offset, r.interleaved))(B.make_rope(tab, 64, 8, True)) == (10, 64, 8, 1)
    for bad in (tab.double(), tab[:, :32], tab.t(), tab.view(-1)):
        with pytest.raises(ValueError):
            B.make_rope(bad, 64)
    for pos in (torch.zeros(4), torch.zeros(8, dtype=torch.int32)[::2], torch.zeros(4, dtype=torch.int64)):
        with pytest.raises(ValueError):
            B.make_rope(tab, 64, positions=pos)
