"""The 4-bit KV cache and the rotating append, as cases to measure.

Operators (include/attn_paged.h):
  attend   attention over a paged cache of E2M1 codes with an E4M3 scale per 16 values
           (attn_run_paged on a plan of kv_dtype ATTN_KV_FP4_E2M1);
  append   new K/V rows quantised into such a cache (attn_append_kv), and into any cache
           with the position rotation of keys and queries on the way (attn_append_kv_rope).
           What the cache then holds of the new tokens is read back as bf16 (attn_read_kv).

`run` computes them in elementary torch operations, or through the framework where `own`
is true.
"""
import math

import numpy as np
import torch

own = False

DV = 128
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEV = "cuda"


def row_bytes(d):
    """Bytes of a 4-bit row of d values: codes, block scales, padding to 16."""
    return (d // 2 + d // 16 + 15) // 16 * 16


def listed():
    def attend(name, **kw):
        c = dict(name=name, op="attend", batch=1, len_min=512, len_max=512, new=1, mixed=False,
                 hq=16, hkv=2, dqk=192, page=128, window=0, sinks=False, len_seed=1)
        return {**c, **kw}

    def append(name, **kw):
        c = dict(name=name, op="append", kv="fp4", rope="none", batch=32, len_min=1024,
                 len_max=4096, new=1, hq=16, hkv=2, dqk=192, page=128, rot=64, rot_off=0, len_seed=1)
        return {**c, **kw}

    return [
        # one short request, one token: what a single user's decode step costs at its start
        attend("attend_tiny", hq=8, hkv=1, page=16),
        # a serving batch of ragged long requests, one token each
        attend("attend_decode", batch=32, len_min=1024, len_max=32767),
        # the same kind of batch on a model with 16 query heads to a KV head, pages of one token
        attend("attend_decode_page1", batch=9, len_min=700, len_max=30001, hq=64, hkv=4, page=1, sinks=True),
        # speculative decoding: eight draft tokens a request checked over a long prefix
        attend("attend_verify", batch=4, len_min=46008, len_max=46008, new=8),
        # a sliding-window layer with sinks, 128/128 heads, decode and verify requests mixed
        attend("attend_window", batch=64, len_min=8192, len_max=8192, new=8, mixed=True, dqk=128,
               window=128, sinks=True),
        # a prompt's later chunk over the tokens already cached
        attend("attend_prefill", len_min=27024, len_max=27024, new=1024, hq=64, hkv=4),
        # the decode step's append: one token a request, latency is what counts
        append("append_decode"),
        # a prompt chunk quantised into the cache, pages that end inside the chunk's tiles
        append("append_prefill", batch=3, new=1365, hkv=4, page=16),
        # decode with rotation of a quarter-to-third of the head, halves paired
        append("rope_decode", kv="fp4", rope="halves", batch=33),
        # a prompt chunk rotated into an 8-bit cache, with its 64 query heads
        append("rope_prefill_fp8", kv="fp8", rope="halves", batch=1, len_min=30096, len_max=30096,
               new=4096, hq=64, hkv=4),
        # neighbours paired, the rotated part behind the unrotated one, a bf16 cache
        append("rope_chunk_bf16", kv="bf16", rope="pairs", batch=7, len_min=900, len_max=2500,
               new=333, page=64, rot_off=128),
        # the whole head rotated into the 4-bit cache
        append("rope_prefill_fp4", kv="fp4", rope="halves", batch=2, len_min=9000, len_max=16000,
               new=2049, hq=32, hkv=8, rot=192),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    hq, hkv = rng.choice([(8, 1), (16, 2), (64, 4), (12, 3), (32, 8), (4, 4), (40, 2)])
    dqk = rng.choice([192, 192, 128])
    page = rng.choice([1, 3, 16, 32, 64, 128])
    c = dict(hq=hq, hkv=hkv, dqk=dqk, page=page, len_seed=rng.randrange(1 << 20))
    if rng.random() < 0.5:
        kind = rng.choice(["decode", "verify", "prefill", "window"])
        new = {"decode": 1, "verify": rng.randint(2, 16), "prefill": _log_int(rng, 33, 900),
               "window": rng.choice([1, 8])}[kind]
        batch = 1 if kind == "prefill" else _log_int(rng, 1, 48)
        keys = 500_000 // hkv                  # keys of the whole batch, all heads: half the largest's
        top = max(new + 1, min(keys // batch, 24_000 if kind == "prefill" else 40_000))
        hi = max(new, _log_int(rng, min(new + 1, top), top))
        return dict(op="attend", batch=batch, len_min=max(new, hi // rng.choice([1, 2, 30])), len_max=hi,
                    new=new, mixed=kind == "window" and new > 1,
                    window=_log_int(rng, 1, 2000) if kind == "window" else 0,
                    sinks=rng.random() < 0.5, **c)
    rope = rng.choice(["none", "halves", "pairs"])
    kv = "fp4" if rope == "none" else rng.choice(["bf16", "fp8", "fp4"])
    rot = 16 * rng.randint(1, dqk // 16)
    rot_off = 8 * rng.randint(0, (dqk - rot) // 8)
    batch = _log_int(rng, 1, 64)
    token = 4 * dqk * (hq if rope != "none" else 0) + 6 * hkv * (dqk + DV)     # bytes, about
    new = _log_int(rng, 1, max(1, min(1500, 180_000_000 // (token * batch))))
    hi = new + _log_int(rng, 1, 3000)
    return dict(op="append", kv=kv, rope=rope, batch=batch, len_min=max(new, hi // 2), len_max=hi, new=new,
                rot=rot, rot_off=rot_off, **c)


def _lengths(case):
    """Requests' lengths and new tokens, from the case alone."""
    rng = np.random.default_rng(case["len_seed"])
    L = rng.integers(case["len_min"], case["len_max"] + 1, size=case["batch"]).astype(np.int64)
    n = np.full(case["batch"], case["new"], np.int64)
    if case.get("mixed"):
        n[::2] = 1
    return L, n


def _key_ranges(case, L, n):
    """First visible key of each request."""
    if case.get("window", 0) > 0:
        return np.maximum(0, L - n - case["window"] + 1)
    return np.zeros_like(L)


def work(case):
    L, n = _lengths(case)
    T, hq, hkv, dqk = int(n.sum()), case["hq"], case["hkv"], case["dqk"]
    index = 4.0 * (2 * len(L) + 1)
    if case["op"] == "attend":
        keys = L - _key_ranges(case, L, n)
        pages = np.ceil(L / case["page"]) - _key_ranges(case, L, n) // case["page"]
        kv = float(keys.sum()) * hkv * (dqk + DV) * (0.5 + 1 / 16)
        flops = 0.0
        for Lb, nb in zip(L.tolist(), n.tolist()):
            i = np.arange(Lb - nb, Lb, dtype=np.float64)
            vis = i + 1 if case["window"] <= 0 else np.minimum(i + 1, case["window"])
            flops += 2.0 * float(vis.sum()) * hq * (dqk + DV)
        return {"bytes": kv + T * hq * (2.0 * dqk + 2.0 * DV + 4) + index + 4 * float(pages.sum()),
                "flops": flops}
    per = {"bf16": 2.0, "fp8": 1.0, "fp4": 0.5 + 1 / 16}[case["kv"]]
    b = T * hkv * (dqk + DV) * (2.0 + per)            # the cache's rows, written
    b += T * hkv * (dqk + DV) * (0.0 if case["kv"] == "bf16" else per + 2.0)   # and read back
    b += index + 4.0 * T
    f = 0.0
    if case["rope"] != "none":
        b += T * (2.0 * hq * 2 * dqk + 4.0 * case["rot"])
        f = 3.0 * T * (hq + hkv) * case["rot"]
    return {"bytes": b, "flops": f}


# --------------------------------------------------------------------------- 4-bit rows, plain

def _quantise(x, scale):
    """fp32 [..., d] -> uint8 rows [..., row_bytes(d)]."""
    d = x.shape[-1]
    y = (x / scale).unflatten(-1, (d // 16, 16))
    s = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float().unsqueeze(-1)
    a = torch.where(sf > 0, y.abs() / sf, torch.zeros_like(y))
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
            + (a > 5.0))
    code = (code + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2)
    packed = code[..., 0::2] + 16 * code[..., 1::2]
    pad = row_bytes(d) - d // 2 - d // 16
    zeros = torch.zeros(*x.shape[:-1], pad, dtype=torch.uint8, device=x.device)
    return torch.cat([packed, s.view(torch.uint8), zeros], -1)


def _values(rows, d, lut):
    """uint8 rows [..., row_bytes(d)] -> fp32 [..., d] (without the tensor's scale); lut: E2M1's 16 values."""
    b = rows[..., : d // 2]
    v = lut[torch.stack([b & 15, b >> 4], -1).flatten(-2).int()]
    s = rows[..., d // 2: d // 2 + d // 16].contiguous().view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (d // 16, 16)) * s.unsqueeze(-1)).flatten(-2)


def _rotate(x, cos, sin, rot, off, rope):
    """x fp32 [T, H, d]; cos, sin [T, 1, rot / 2]."""
    part = x[..., off: off + rot]
    if rope == "halves":
        x1, x2 = part[..., : rot // 2], part[..., rot // 2:]
        turned = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
    else:
        x1, x2 = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2)
    return torch.cat([x[..., :off], turned, x[..., off + rot:]], -1)


# --------------------------------------------------------------------------- inputs

def _cache(g, slots, hkv, d, scale, kv, std):
    """Rows of a pool of `slots` slots, filled as earlier appends left them."""
    x = torch.randn(slots, hkv, d, generator=g, device=DEV) * std
    if kv == "bf16":
        return x.bfloat16()
    if kv == "fp8":
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return _quantise(x, scale)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    L, n = _lengths(case)
    B, P, hq, hkv, dqk = case["batch"], case["page"], case["hq"], case["hkv"], case["dqk"]
    T = int(n.sum())
    pages = -(-L // P)
    num_pages = int(pages.sum()) + 2
    stride = int(pages.max())
    perm = torch.randperm(num_pages, generator=g, device=DEV).int()
    col = torch.arange(stride, device=DEV)
    first = torch.tensor(np.concatenate([[0], np.cumsum(pages)[:-1]]), device=DEV)
    count = torch.tensor(pages, device=DEV)
    table = perm[(first[:, None] + col).clamp(max=num_pages - 1)]
    table = torch.where(col < count[:, None], table, perm[-1]).contiguous()
    qo = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
    lens = torch.tensor(L, dtype=torch.int32, device=DEV)
    kv = case.get("kv", "fp4")
    top = {"bf16": None, "fp8": 448.0, "fp4": 6.0 * 448.0}[kv]
    ks, vs = (1.0, 1.0) if top is None else (float(np.float32(5.4371 / top)), float(np.float32(6.0193 / top)))
    s = dict(case=case, L=L, n=n, T=T, q=torch.randn(T, hq, dqk, generator=g, device=DEV).bfloat16(),
             page_table=table, qo=qo, lens=lens,
             lut=torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV), k_scale=ks, v_scale=vs, num_pages=num_pages)
    # the request and the position of every new token
    req = torch.tensor(np.repeat(np.arange(B), n), device=DEV)
    pos = torch.tensor(np.concatenate([np.arange(a - b, a) for a, b in zip(L, n)]), device=DEV)
    s["req"], s["pos"] = req, pos
    slot = lambda d, std, sc: _cache(g, num_pages * P, hkv, d, sc, kv, std)  # noqa: E731
    s["k_cache"] = slot(dqk, 0.8, ks).view(num_pages, P, hkv, -1)
    s["v_cache"] = slot(DV, 1.0, vs).view(num_pages, P, hkv, -1)
    if case["op"] == "attend":
        # slots behind a request's last key, and pages nobody owns, were never written
        key = torch.arange(stride * P, device=DEV)
        sl = (table.long()[:, key // P] * P + key % P)
        used = torch.zeros(num_pages * P, dtype=torch.bool, device=DEV)
        used[sl[key < lens[:, None]]] = True
        s["k_cache"].view(num_pages * P, -1)[~used] = 0xFF
        s["v_cache"].view(num_pages * P, -1)[~used] = 0xFF
        s["sinks"] = torch.randn(hq, generator=g, device=DEV) if case["sinks"] else None
        s["scale"] = 1.0 / math.sqrt(dqk)
        lo = _key_ranges(case, L, n)
        s["lo"] = torch.tensor(lo, device=DEV)
        s["span"] = int((L - lo).max())
        s["nmax"] = int(n.max())
    else:
        s["k_new"] = (torch.randn(T, hkv, dqk, generator=g, device=DEV) * 0.8).bfloat16()
        s["v_new"] = torch.randn(T, hkv, DV, generator=g, device=DEV).bfloat16()
        if case["rope"] != "none":
            half = case["rot"] // 2
            inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
            ang = torch.arange(int(L.max()) + 1, dtype=torch.float64, device=DEV)[:, None] * inv
            s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], -1).float().contiguous()
    if own:
        from asymmetric_kv_paged_gb300 import binding as B_
        kinds = {"bf16": B_.ATTN_KV_BF16, "fp8": B_.ATTN_KV_FP8_E4M3, "fp4": B_.ATTN_KV_FP4_E2M1}
        prob, keep = B_.make_problem(
            batch=B, num_q_heads=hq, num_kv_heads=hkv, page_size=P, num_pages=num_pages,
            page_table_stride=stride, kv_dtype=kinds[kv], window=case.get("window", 0),
            has_sinks=case.get("sinks", False), qo_indptr=np.concatenate([[0], np.cumsum(n)]),
            seq_lens=L, head_dim_qk=dqk)
        s["plan"] = B_.attn_plan(prob, torch.cuda.current_device(), keep)
        s["workspace"] = torch.empty(max(1, s["plan"].workspace_bytes), dtype=torch.uint8, device=DEV)
        bf = dict(dtype=torch.bfloat16, device=DEV)
        if case["op"] == "attend":
            s["out"] = torch.empty(T, hq, DV, **bf)
            s["lse"] = torch.empty(T, hq, dtype=torch.float32, device=DEV)
        else:
            s["k_read"], s["v_read"] = torch.empty(T, hkv, dqk, **bf), torch.empty(T, hkv, DV, **bf)
            if case["rope"] != "none":
                s["q_out"] = torch.empty(T, hq, dqk, **bf)
                s["rope"] = B_.make_rope(s["cos_sin"], case["rot"], rot_offset=case["rot_off"],
                                         interleaved=case["rope"] == "pairs")
    return s


# --------------------------------------------------------------------------- one pass

def _attend_plain(s):
    c = s["case"]
    hq, hkv, dqk, P = c["hq"], c["hkv"], c["dqk"], c["page"]
    G, B, nmax, span = hq // hkv, c["batch"], s["nmax"], s["span"]
    key = s["lo"][:, None] + torch.arange(span, device=DEV)                    # [B, span]
    inside = key < s["lens"][:, None]
    kc = torch.where(inside, key, s["lo"][:, None])
    slot = s["page_table"].long().gather(1, kc // P) * P + kc % P
    K = _values(s["k_cache"].flatten(0, 1)[slot], dqk, s["lut"]) * s["k_scale"]   # [B, span, hkv, dqk]
    V = _values(s["v_cache"].flatten(0, 1)[slot], DV, s["lut"]) * s["v_scale"]
    row = s["qo"][:-1, None].long() + torch.arange(nmax, device=DEV)           # [B, nmax] flat tokens
    n = (s["qo"][1:] - s["qo"][:-1]).long()
    live = torch.arange(nmax, device=DEV) < n[:, None]
    q = s["q"][torch.where(live, row, torch.zeros_like(row))].float()          # [B, nmax, hq, dqk]
    q = q.view(B, nmax, hkv, G, dqk).permute(0, 2, 1, 3, 4).reshape(B, hkv, nmax * G, dqk)
    S = (q @ K.permute(0, 2, 3, 1)) * s["scale"]                               # [B, hkv, nmax * G, span]
    i = (s["lens"].long() - n)[:, None] + torch.arange(nmax, device=DEV)       # [B, nmax]
    see = inside[:, None] & (key[:, None] <= i[..., None])
    if c["window"] > 0:
        see = see & (key[:, None] > i[..., None] - c["window"])
    see = see[:, None, :, None].expand(B, 1, nmax, G, span).reshape(B, 1, nmax * G, span)
    S = S.masked_fill_(~see, -math.inf)
    m = S.amax(-1, keepdim=True)
    if s["sinks"] is not None:
        sink = s["sinks"].view(1, hkv, 1, G).expand(B, hkv, nmax, G).reshape(B, hkv, nmax * G, 1)
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = S.sub_(m).exp_()
    z = p.sum(-1, keepdim=True)
    if s["sinks"] is not None:
        z = z + (sink - m).exp()
    o = (p @ V.permute(0, 2, 1, 3)) / z
    lse = (m + z.log()).squeeze(-1)
    o = o.view(B, hkv, nmax, G, DV).permute(0, 2, 1, 3, 4).reshape(B, nmax, hq, DV)
    lse = lse.view(B, hkv, nmax, G).permute(0, 2, 1, 3).reshape(B, nmax, hq)
    return {"out": o[live].bfloat16(), "lse": lse[live]}


def _append_plain(s):
    c = s["case"]
    P, kv = c["page"], c["kv"]
    k, v = s["k_new"].float(), s["v_new"].float()
    out = {}
    if c["rope"] != "none":
        cs = s["cos_sin"][s["pos"]][:, None]
        cos, sin = cs[..., : c["rot"] // 2], cs[..., c["rot"] // 2:]
        k = _rotate(k, cos, sin, c["rot"], c["rot_off"], c["rope"])
        out["q"] = _rotate(s["q"].float(), cos, sin, c["rot"], c["rot_off"], c["rope"]).bfloat16()
    slot = s["page_table"].long()[s["req"], s["pos"] // P] * P + s["pos"] % P
    kc, vc = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    if kv == "bf16":
        kc[slot], vc[slot] = k.bfloat16(), v.bfloat16()
        return {**out, "k": s["k_cache"], "v": s["v_cache"]}
    if kv == "fp8":
        put = lambda x, sc: (x / sc).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)  # noqa: E731
        kc[slot], vc[slot] = put(k, s["k_scale"]), put(v, s["v_scale"])
        get = lambda r, d: r.view(torch.float8_e4m3fn).float()  # noqa: E731
    else:
        kc[slot], vc[slot] = _quantise(k, s["k_scale"]), _quantise(v, s["v_scale"])
        get = lambda r, d: _values(r, d, s["lut"])  # noqa: E731
    out["k"] = (get(kc[slot], c["dqk"]) * s["k_scale"]).bfloat16()
    out["v"] = (get(vc[slot], DV) * s["v_scale"]).bfloat16()
    return out


def run(s):
    c = s["case"]
    if not own:
        return _attend_plain(s) if c["op"] == "attend" else _append_plain(s)
    from asymmetric_kv_paged_gb300 import binding as B_
    if c["op"] == "attend":
        B_.attn_run_paged(s["plan"], s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"],
                          s["qo"], s["sinks"], c["window"], s["scale"], s["k_scale"], s["v_scale"],
                          s["out"], s["lse"], s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    out = {}
    if c["rope"] == "none":
        B_.attn_append_kv(s["plan"], s["k_new"], s["v_new"], s["k_cache"], s["v_cache"], s["page_table"],
                          s["lens"], s["qo"], s["k_scale"], s["v_scale"])
    else:
        B_.attn_append_kv_rope(s["plan"], s["rope"], s["q"], s["k_new"], s["v_new"], s["q_out"],
                               s["k_cache"], s["v_cache"], s["page_table"], s["lens"], s["qo"],
                               s["k_scale"], s["v_scale"])
        out["q"] = s["q_out"]
    if c["kv"] == "bf16":
        return {**out, "k": s["k_cache"], "v": s["v_cache"]}
    B_.attn_read_kv(s["plan"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"], s["qo"],
                    s["k_read"], s["v_read"], s["k_scale"], s["v_scale"])
    return {**out, "k": s["k_read"], "v": s["v_read"]}


# --------------------------------------------------------------------------- 64 bits

def _nearest(a, table):
    """Index of the nearest value of an increasing table, ties to the even index."""
    mid = (table[1:] + table[:-1]) / 2
    i = torch.searchsorted(mid, a.contiguous())
    tie = (i < mid.numel()) & (mid[i.clamp(max=mid.numel() - 1)] == a) & (i % 2 == 1)
    return i + tie


def _e4m3_table():
    v = [m / 8 * 2.0 ** -6 for m in range(8)]
    v += [(1 + m / 8) * 2.0 ** (e - 7) for e in range(1, 16) for m in range(8)]
    return torch.tensor(v[:-1], dtype=torch.float64, device=DEV)


def _decode64(rows, d):
    """The same rows from the format's bit fields, in 64 bits."""
    r = rows.long()
    code = torch.stack([r[..., : d // 2] % 16, r[..., : d // 2] // 16], -1).flatten(-2)
    e, m = code // 2 % 4, code % 2
    mag = torch.where(e == 0, m * 0.5, (1 + m * 0.5) * torch.exp2((e - 1).double()))
    val = torch.where(code >= 8, -mag, mag)
    sc = _e4m3_table()[r[..., d // 2: d // 2 + d // 16].clamp(max=126)]
    return val * sc.repeat_interleave(16, -1)


def _round64(x, scale, kv):
    """What a cache holds of x, in 64 bits."""
    if kv == "bf16":
        return x
    y = x / scale
    t8 = _e4m3_table()
    if kv == "fp8":
        return torch.sign(y) * t8[_nearest(y.abs(), t8)] * scale
    b = y.unflatten(-1, (-1, 16))
    s = t8[_nearest(b.abs().amax(-1) / 6, t8)].unsqueeze(-1)
    t4 = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    z = torch.where(s > 0, b.abs() / s, torch.zeros_like(b))
    return (torch.sign(b) * t4[_nearest(z, t4)] * s).flatten(-2) * scale


def _attend64(s):
    c = s["case"]
    G, P = c["hq"] // c["hkv"], c["page"]
    out = torch.zeros(s["T"], c["hq"], DV, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["T"], c["hq"], dtype=torch.float64, device=DEV)
    t0 = 0
    for b, (L, n) in enumerate(zip(s["L"].tolist(), s["n"].tolist())):
        j = torch.arange(int(s["lo"][b]), L, device=DEV)
        slot = s["page_table"][b].long()[j // P] * P + j % P
        i = torch.arange(L - n, L, device=DEV)[:, None]
        see = j <= i
        if c["window"] > 0:
            see &= j > i - c["window"]
        for g in range(c["hkv"]):
            K = _decode64(s["k_cache"].flatten(0, 1)[slot, g], c["dqk"]) * s["k_scale"]
            V = _decode64(s["v_cache"].flatten(0, 1)[slot, g], DV) * s["v_scale"]
            q = s["q"][t0:t0 + n, g * G:(g + 1) * G].double().transpose(0, 1)
            S = torch.where(see, (q @ K.T) * s["scale"], -math.inf)            # [G, n, keys]
            if s["sinks"] is not None:
                sk = s["sinks"][g * G:(g + 1) * G].double().view(G, 1, 1)
                Z = torch.logsumexp(torch.cat([S, sk.expand(G, n, 1)], -1), -1)
            else:
                Z = torch.logsumexp(S, -1)
            out[t0:t0 + n, g * G:(g + 1) * G] = (torch.exp(S - Z[..., None]) @ V).transpose(0, 1)
            lse[t0:t0 + n, g * G:(g + 1) * G] = Z.T
        t0 += n
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attend":
        return _attend64(s)
    out = {}
    k, v = s["k_new"].double(), s["v_new"].double()
    if case["rope"] != "none":
        half, off = case["rot"] // 2, case["rot_off"]
        w = torch.view_as_complex(torch.stack([s["cos_sin"][s["pos"], :half],
                                               s["cos_sin"][s["pos"], half:]], -1).double())[:, None]
        at = torch.arange(half, device=DEV)
        i1, i2 = (off + at, off + half + at) if case["rope"] == "halves" else (off + 2 * at, off + 2 * at + 1)

        def turn(x):
            y = x.clone()
            z = torch.complex(x[..., i1], x[..., i2]) * w
            y[..., i1], y[..., i2] = z.real, z.imag
            return y

        k, out["q"] = turn(k), turn(s["q"].double())
    if case["kv"] == "bf16":
        P = case["page"]
        slot = s["page_table"].long()[s["req"], s["pos"] // P] * P + s["pos"] % P
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        kc.flatten(0, 1)[slot], vc.flatten(0, 1)[slot] = k, v
        return {**out, "k": kc, "v": vc}
    return {**out, "k": _round64(k, s["k_scale"], case["kv"]), "v": _round64(v, s["v_scale"], case["kv"])}
