"""attn_select_blocks where the heads of one group lie up to 2^247 apart: the small head's share of a
score underflows as fp32 rounds it, alike for few tokens and for chunks of them."""
import numpy as np
import pytest

import sparse_plain as P_
from asymmetric_kv_paged_gb300 import workloads as W

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from test_gpu_select import random_bounds, run, setup  # noqa: E402


def scores(q, recs, d):
    """A group's scores as fp32 holds them: d(h, c) * 2^(e_h - max e), then the largest times 2^(e_c),
    each product rounded once.  float64 holds both products of such numbers exactly."""
    r = recs.view(np.int8).astype(np.float64)
    hi, lo, ec = r[:, :d], r[:, d:2 * d], r[:, 2 * d]
    exps = [P_.exponent(np.abs(x).max(), hi=121) for x in q]
    top = np.full(len(recs), -np.inf, np.float32)
    for x, e in zip(q, exps):
        qi = np.rint(x / 2.0 ** e)
        dot = np.maximum(qi * hi, qi * lo).sum(1)
        top = np.maximum(top, (dot * 2.0 ** (e - max(exps))).astype(np.float32))
    return (top.astype(np.float64) * 2.0 ** ec).astype(np.float32)


@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("dqk", [192, 128])
@pytest.mark.parametrize("apart", [17, 100, 122, 123, 140, 149, 150, 155, 165, 166, 170, 172, 200, 247])
def test_heads_far_apart_in_one_group(n, dqk, apart):
    """A large head whose scores are all negative and a small one whose scores are positive: the
    small one decides, until nothing of it is left and all blocks are alike."""
    from asymmetric_kv_paged_gb300 import binding as B
    w, dw = setup([3000], [n], 16, 2, 64, dqk)
    rng = np.random.default_rng(apart)
    bounds = random_bounds(rng, w, 64).view(np.int8)
    bounds[..., :dqk] = -rng.integers(1, 60, bounds.shape[:-1] + (dqk,))
    bounds[..., dqk:2 * dqk] = bounds[..., :dqk] - rng.integers(0, 60, bounds.shape[:-1] + (dqk,))
    bounds[..., 2 * dqk] = rng.integers(-3, 4, bounds.shape[:-1])
    small = -126 + (247 - apart) // 2
    q = np.zeros((n, 16, dqk), np.float32)
    # whole numbers of 64 to 127: e_h is the power of two (at most 127 * 2^121, a finite bf16)
    q[:, 0::8] = rng.integers(64, 128, (n, 2, dqk)) * np.float32(2.0) ** (small + apart)
    q[:, 5::8] = -rng.integers(64, 128, (n, 2, dqk)) * np.float32(2.0) ** small
    qb = W.bf16_bits(q)
    qv = W.bf16_values(qb).astype(np.float64)
    for h in range(16):
        if h % 8 not in (0, 5):
            qb[:, h] = qb[:, h - h % 8]                            # the other heads repeat the large one
            qv[:, h] = qv[:, h - h % 8]
    got = run(w, dw, qb, bounds.view(np.uint8), 64, 12, 1, 2)
    assert B.attn_get_device_error(dw.plan) == 0
    flat = bounds.view(np.uint8).reshape(-1, 2, bounds.shape[-1])
    at = P_.slots(w, 0, np.arange(47) * 64) // 64
    alike = []
    for tok in range(n):
        own = (3000 - n + tok) // 64
        for g in range(2):
            s = scores(qv[tok, 8 * g:8 * g + 8], flat[at[:own + 1], g], dqk)
            want = P_.choose(s, own, 12, 1, 2)
            assert np.array_equal(got[tok, g], want), (tok, g)
            alike.append(len(set(s[1:own - 1])) == 1)
    # 2^22 * 2^-172 and less is nothing in fp32; up to 2^-149 every unit of d counts
    assert all(alike) if apart >= 172 else not any(alike) if apart <= 149 else True
