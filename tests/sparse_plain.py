"""Plain 64-bit forms of the operators of attention over selected blocks, for the tests.

Everything is read literally from include/attn_paged.h: bounds records from the cached
values, block lists from the records, attention over the listed keys one row at a time.
"""
import math

import numpy as np

from asymmetric_kv_paged_gb300 import workloads as W


def cached_values(rows, d, kv):
    """Cached rows -> float64 values without the tensor's scale (the E4M3 and scale NaNs too)."""
    if kv == "bf16":
        return W.bf16_values(rows).astype(np.float64)
    if kv == "fp4":
        return W.fp4_values(rows, d).astype(np.float64)
    import torch
    return torch.from_numpy(np.ascontiguousarray(rows)).view(torch.float8_e4m3fn).double().numpy()


def exponent(amax, lo=-126, hi=122):
    if amax == 0:
        return 0
    e = lo
    while amax > 127.0 * 2.0 ** e:
        e += 1
    return min(e, hi)


def record(rows, bytes_):
    """Rows of one block and head [block, d] float64 -> its record."""
    d = rows.shape[1]
    rec = np.zeros(bytes_, np.int8)
    if not np.isfinite(rows).all():
        rec[2 * d] = 127
        return rec.view(np.uint8)
    e = exponent(np.abs(rows).max())
    rec[:d] = np.ceil(rows.max(0) / 2.0 ** e)
    rec[d:2 * d] = np.floor(rows.min(0) / 2.0 ** e)
    rec[2 * d] = e
    return rec.view(np.uint8)


def slots(w, b, pos):
    pos = np.asarray(pos, np.int64)
    return w.page_table[b][pos // w.page_size].astype(np.int64) * w.page_size + pos % w.page_size


def update_bounds(w, bounds, block, k_cache, seq_lens, indptr):
    """The bounds array [num_pages, P / block, hkv, row] after the rows of indptr."""
    out = bounds.copy()
    flat = k_cache.reshape(-1, *k_cache.shape[2:])
    for b, L in enumerate(np.asarray(seq_lens).tolist()):
        m = int(indptr[b + 1] - indptr[b])
        for pos in range(L - m, L):
            if (pos + 1) % block:
                continue
            s = int(slots(w, b, pos + 1 - block))
            vals = cached_values(flat[s:s + block], w.dqk, w.kv_dtype)
            for g in range(w.hkv):
                out.reshape(-1, w.hkv, out.shape[-1])[s // block, g] = record(vals[:, g], out.shape[-1])
    return out


def scores(q, recs, d):
    """q float64 [heads, d] of one group; recs [blocks, row] uint8 -> float64 [blocks]."""
    r = recs.view(np.int8).astype(np.float64)
    hi, lo, e = r[:, :d], r[:, d:2 * d], r[:, 2 * d]
    top = np.full(len(recs), -np.inf)
    heads = [x for x in q if np.isfinite(x).all()]
    exps = [exponent(np.abs(x).max(), hi=121) for x in heads]
    for x, eh in zip(heads, exps):
        qi = np.rint(x / 2.0 ** eh)
        dot = np.maximum(qi * hi, qi * lo).sum(1)
        top = np.maximum(top, dot * 2.0 ** (eh - max(exps)))
    with np.errstate(invalid="ignore"):
        return np.where(e == 127, np.inf, top * 2.0 ** np.where(e == 127, 0, e))


def choose(score, own, take, first, last):
    """One list: score [own + 1] (the forced blocks' entries are not looked at)."""
    c = np.arange(own + 1)
    forced = (c < first) | (c > own - last)
    rest = sorted(c[~forced], key=lambda i: (-score[i], i))
    picked = sorted(list(c[forced]) + rest[:max(0, take - int(forced.sum()))])
    if own < take:
        picked = list(c)
    return np.array(picked + [-1] * (take - len(picked)), np.int32)


def select(w, q, bounds, block, take, first, last, seq_lens=None):
    """block_idx [T, hkv, take]; q: bf16 bits."""
    seq_lens = w.seq_lens if seq_lens is None else seq_lens
    qv = W.bf16_values(q).astype(np.float64)
    G = w.hq // w.hkv
    out = np.full((w.total_q, w.hkv, take), -1, np.int32)
    flat = bounds.reshape(-1, w.hkv, bounds.shape[-1])
    for b, L in enumerate(np.asarray(seq_lens).tolist()):
        t0, t1 = int(w.qo_indptr[b]), int(w.qo_indptr[b + 1])
        nb = (L - 1) // block + 1
        at = slots(w, b, np.arange(nb) * block) // block if t1 > t0 else None
        for tok in range(t0, t1):
            own = (L - t1 + tok) // block
            for g in range(w.hkv):
                s = scores(qv[tok, g * G:(g + 1) * G], flat[at[:own + 1], g], w.dqk)
                out[tok, g] = choose(s, own, take, first, last)
    return out


def attend(w, q, block, block_idx, sinks=None, seq_lens=None, k_cache=None, v_cache=None):
    """out, lse, |v|-weighted out, the largest sum of |q k| scale, and the sum of |v|, all float64."""
    seq_lens = w.seq_lens if seq_lens is None else seq_lens
    k_cache = w.k_cache if k_cache is None else k_cache
    v_cache = w.v_cache if v_cache is None else v_cache
    qv = W.bf16_values(q).astype(np.float64)
    G, D = w.hq // w.hkv, w.dqk
    ks, vs = (1.0, 1.0) if w.kv_dtype == "bf16" else (w.k_scale, w.v_scale)
    T = w.total_q
    out, mag = np.zeros((T, w.hq, 128)), np.zeros((T, w.hq, 128))
    lse, smag, vsum = np.full((T, w.hq), -np.inf), np.zeros((T, w.hq)), np.zeros((T, w.hq, 128))
    kf, vf = k_cache.reshape(-1, *k_cache.shape[2:]), v_cache.reshape(-1, *v_cache.shape[2:])
    for b, L in enumerate(np.asarray(seq_lens).tolist()):
        t0, t1 = int(w.qo_indptr[b]), int(w.qo_indptr[b + 1])
        for tok in range(t0, t1):
            i = L - t1 + tok
            for g in range(w.hkv):
                blocks = sorted({int(c) for c in block_idx[tok, g] if 0 <= c <= i // block})
                pos = np.array([j for c in blocks for j in range(c * block, min((c + 1) * block, i + 1))], np.int64)
                h = slice(g * G, (g + 1) * G)
                sink = None if sinks is None else sinks[h].astype(np.float64)
                if not len(pos):
                    if sink is not None:
                        lse[tok, h] = sink
                    continue
                s = slots(w, b, pos)
                K = cached_values(kf[s, g], D, w.kv_dtype) * ks
                V = cached_values(vf[s, g], 128, w.kv_dtype) * vs
                S = qv[tok, h] @ K.T * w.softmax_scale
                smag[tok, h] = (np.abs(qv[tok, h]) @ np.abs(K.T)).max(1) * w.softmax_scale
                vsum[tok, h] = np.abs(V).sum(0)
                m = S.max(1) if sink is None else np.maximum(S.max(1), sink)
                p = np.exp(S - m[:, None])
                z = p.sum(1) + (0 if sink is None else np.exp(sink - m))
                out[tok, h], mag[tok, h] = p @ V / z[:, None], p @ np.abs(V) / z[:, None]
                lse[tok, h] = m + np.log(z)
    return out, lse, mag, smag, vsum


def assert_close(got_out, got_lse, ref, kv, what=""):
    """Kernel outputs against attend()'s.  The weights are held in bf16 (8 bits) or fp16 (11),
    half a step each relative to the weight; the scores are fp32 sums of D products, each
    addition off by at most a step of 2^-23 of what was added up in magnitude; e^x turns that
    into a relative error of every weight and of their sum; the result is rounded to bf16.

    fp16 weights are held as 2^7 w, w <= 1 relative to the running maximum.  Below 2^-14 fp16's
    steps stay at 2^-24, so that a weight under 2^-21 is off by up to 2^-25 / 2^7 = 2^-32 of the
    maximum's weight instead of 2^-11 of itself: over a row at most 2^-32 sum |v| (the sum of the
    weights it is divided by is at least the maximum's, 1).  A row whose large weights all meet
    values of exactly zero consists of such weights."""
    out, lse, mag, smag, vsum = ref
    weight = 2.0 ** -8 if kv == "bf16" else 2.0 ** -11
    s_err = 200 * 2.0 ** -23 * smag + 2.0 ** -20                # and ex2's, log2's few steps
    tol = (1.01 * weight + 2 * s_err)[..., None] * mag + 2.0 ** -8 * np.abs(out) + 1e-30
    if kv != "bf16":
        tol += 2.0 ** -32 * vsum
    err = np.abs(got_out - out)
    assert np.all(err <= tol), f"{what}: out off by {np.max(err / tol):.3g} of the tolerance"
    live = np.isfinite(lse)
    assert np.array_equal(np.isfinite(got_lse), live), what
    e = np.abs(got_lse[live] - lse[live])
    t = s_err[live] + 2.0 ** -22 * np.abs(lse[live]) + 2.0 ** -20
    assert np.all(e <= t), f"{what}: lse off by {np.max(e / t, initial=0):.3g} of the tolerance"
    assert math.isinf(-lse[~live].max(initial=-math.inf))
