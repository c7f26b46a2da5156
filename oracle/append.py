"""FP64/CPU oracle for the KV-append step (numpy), test infrastructure only.

The tests and the benchmark's CPU leg are its only callers; the product path
never imports it, and it imports nothing from the product package.

Definition (the step before attention, model card
MiMo-V2.6-Flash-RL-FP8KV-W4A8-2x-RTX-PRO-6000, "What the kernels do": an FP8
E4M3 KV cache with per-tensor scales): request b's new token t sits at
position i = seq_lens[b] - n_b + t; its K and V rows go to page
page_table[b][i // P], offset i % P, every KV head.  BF16 caches take the
bf16 bits unchanged.  FP8 caches take the E4M3 code nearest to x / scale,
where x is the bf16 value and the quotient is the fp32 IEEE quotient (the
precision the kernel decides in); ties go to the code with an even mantissa,
magnitudes beyond the largest finite E4M3 value (448) saturate to it.

The encoder is the definition read literally: it looks for the nearest value
among all finite E4M3 codes, decoded from the format (sign, 4-bit exponent
with bias 7, 3-bit mantissa, subnormals below 2^-6; 0x7F/0xFF are NaN).
Parity pins: tests/test_oracle_pins.py (append section).
"""
from __future__ import annotations

import numpy as np


def e4m3_decode(code: int) -> float:
    s = -1.0 if code & 0x80 else 1.0
    e = (code >> 3) & 0xF
    m = code & 0x7
    if e == 0xF and m == 0x7:
        return float("nan")
    if e == 0:
        return s * (m / 8.0) * 2.0 ** -6
    return s * (1.0 + m / 8.0) * 2.0 ** (e - 7)


# the 127 non-negative finite codes 0x00..0x7E, in increasing value order
_POS_CODES = np.arange(0x7F, dtype=np.int64)
_POS_VALUES = np.array([e4m3_decode(int(c)) for c in _POS_CODES], dtype=np.float64)


def e4m3_encode(x: float) -> int:
    """Nearest E4M3 code to x, ties to even mantissa, saturating at 448."""
    if np.isnan(x):
        return 0x7F
    sign = 0x80 if np.signbit(x) else 0
    a = abs(float(x))
    if a >= _POS_VALUES[-1]:
        return sign | 0x7E
    d = np.abs(_POS_VALUES - a)
    best = np.flatnonzero(d == d.min())
    if best.size > 1:                      # a tie between two neighbours
        best = best[(_POS_CODES[best] & 1) == 0]
    return sign | int(_POS_CODES[best[0]])


def bf16_to_f32(bits: np.ndarray) -> np.ndarray:
    return (np.asarray(bits, np.uint16).astype(np.uint32) << 16).view(np.float32)


# the eight E2M1 magnitudes, in code order (even codes have an even mantissa)
_E2M1_VALUES = np.array([m * 0.5 if e == 0 else (1 + m * 0.5) * 2.0 ** (e - 1)
                         for e in range(4) for m in range(2)], dtype=np.float64)


def e2m1_encode(x: float) -> int:
    """Nearest E2M1 code to x, ties to even mantissa, saturating at 6."""
    sign = 8 if np.signbit(x) else 0
    d = np.abs(_E2M1_VALUES - min(abs(float(x)), 6.0))
    best = np.flatnonzero(d == d.min())
    if best.size > 1:
        best = best[(best & 1) == 0]
    return sign | int(best[0])


def fp4_row(x: np.ndarray, scale: float) -> np.ndarray:
    """One 4-bit cache row (codes, block scales, zero padding) of the fp32 row x:
    y = x / scale; per 16 values the block scale E4M3(max|y| / 6), then the E2M1
    code of y / block scale; every quotient the fp32 IEEE one."""
    d = x.size
    out = np.zeros((d // 2 + d // 16 + 15) // 16 * 16, np.uint8)
    with np.errstate(over="ignore", invalid="ignore"):
        y = (x.astype(np.float32) / np.float32(scale)).astype(np.float32)
        for c in range(d // 16):
            blk = y[16 * c:16 * c + 16]
            code = e4m3_encode(np.abs(blk).max() / np.float32(6.0))
            out[d // 2 + c] = code
            s = np.float32(e4m3_decode(code))
            if np.isnan(s):                      # the codes under a NaN scale mean nothing
                continue
            q = blk / s if s > 0 else np.copysign(np.float32(0), blk)
            codes = [e2m1_encode(v) for v in q]
            for i in range(8):
                out[8 * c + i] = codes[2 * i] | codes[2 * i + 1] << 4
    return out


def fp4_row_values(row: np.ndarray, d: int) -> np.ndarray:
    """The float64 values a 4-bit row stands for, from the format's bit fields."""
    out = np.empty(d)
    for i in range(d):
        code = (int(row[i // 2]) >> (4 * (i % 2))) & 15
        v = _E2M1_VALUES[code & 7] * (-1.0 if code & 8 else 1.0)
        out[i] = v * e4m3_decode(int(row[d // 2 + i // 16]))
    return out


def rotate(x: np.ndarray, cos_sin: np.ndarray, rot: int, off: int, interleaved: bool) -> np.ndarray:
    """fp32 rows x [..., d] rotated by the table rows cos_sin [..., rot]: pair i is dims
    (off + i, off + rot/2 + i), or (off + 2i, off + 2i + 1); every product, sum and
    difference is one fp32 operation."""
    x = np.array(x, np.float32)
    half = rot // 2
    c, s = np.float32(cos_sin[..., :half]), np.float32(cos_sin[..., half:])
    i = np.arange(half)
    a, b = (off + 2 * i, off + 2 * i + 1) if interleaved else (off + i, off + half + i)
    x1, x2 = x[..., a].copy(), x[..., b].copy()
    x[..., a] = (x1 * c) - (x2 * s)
    x[..., b] = (x2 * c) + (x1 * s)
    return x


def f32_to_bf16(x: np.ndarray) -> np.ndarray:
    """bf16 bits of fp32 values, nearest even."""
    u = np.ascontiguousarray(x, np.float32).view(np.uint32).astype(np.uint64)
    r = ((u + 0x7FFF + ((u >> 16) & 1)) >> 16).astype(np.uint16)
    return np.where(np.isnan(x), np.uint16(0x7FFF), r)


def append_rows(rows_k, rows_v, k_cache, v_cache, page_table, seq_lens, qo_indptr, kv_dtype: str,
                k_scale: float = 1.0, v_scale: float = 1.0):
    """append_kv for fp32 rows [total_q, Hkv, D] (rotated keys) into a cache of any
    type; returns the caches after it."""
    kc, vc = np.array(k_cache, copy=True), np.array(v_cache, copy=True)
    num_pages, P = kc.shape[0], kc.shape[1]

    def stored(row, scale):                      # [Hkv, D] fp32 -> [Hkv, row]
        if kv_dtype == "bf16":
            return f32_to_bf16(row)
        if kv_dtype == "fp8":
            return np.vectorize(e4m3_encode, otypes=[np.uint8])(row / np.float32(scale))
        return np.stack([fp4_row(r, scale) for r in row])

    for b in range(len(seq_lens)):
        q0, q1 = int(qo_indptr[b]), int(qo_indptr[b + 1])
        for t in range(q0, q1):
            i = int(seq_lens[b]) - (q1 - t)
            page = int(page_table[b][i // P])
            if 0 <= page < num_pages:
                kc[page, i % P] = stored(rows_k[t], k_scale)
                vc[page, i % P] = stored(rows_v[t], v_scale)
    return kc, vc


def append_kv(k_new, v_new, k_cache, v_cache, page_table, seq_lens, qo_indptr,
              kv_dtype: str, k_scale: float = 1.0, v_scale: float = 1.0):
    """Returns (k_cache, v_cache) after the append, as new arrays, and the number
    of tokens skipped for an out-of-pool page id.  k_new/v_new: uint16 (bf16 bits)
    [total_q, Hkv, D]; caches: uint16 (bf16) or uint8 (E4M3) [pages, P, Hkv, D]."""
    kc = np.array(k_cache, copy=True)
    vc = np.array(v_cache, copy=True)
    num_pages, P = kc.shape[0], kc.shape[1]
    skipped = 0
    for b in range(len(seq_lens)):
        q0, q1 = int(qo_indptr[b]), int(qo_indptr[b + 1])
        n = q1 - q0
        for t in range(n):
            i = int(seq_lens[b]) - n + t
            page = int(page_table[b][i // P])
            if page < 0 or page >= num_pages:
                skipped += 1
                continue
            for cache, new, scale in ((kc, k_new, k_scale), (vc, v_new, v_scale)):
                row = np.asarray(new[q0 + t])
                if kv_dtype == "bf16":
                    cache[page, i % P] = row
                else:
                    q = bf16_to_f32(row) / np.float32(scale)      # fp32 IEEE quotient
                    cache[page, i % P] = np.vectorize(e4m3_encode, otypes=[np.uint8])(q)
    return kc, vc, skipped
