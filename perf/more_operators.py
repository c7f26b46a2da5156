"""Attention over selected blocks and rotation by positions of several axes, as cases to measure.

Operators (include/attn_paged.h):
  mrope    new K/V rows into a paged cache, keys and queries rotated by positions of several
           axes (attn_append_kv_mrope); what an 8- or 4-bit cache then holds is read back
           (attn_read_kv);
  bounds   the smallest and largest key of every completed block of the cache, per dimension,
           in 8 bits (attn_update_bounds), and read back as bf16 (attn_read_bounds);
  select   for every new token and KV head the blocks to attend to: the first, the last and
           those whose bound on the scores is largest (attn_select_blocks);
  sparse   attention of every new token over its own list of blocks (attn_run_sparse).

`run` computes them in elementary torch operations, or through the framework where `own` is
true.
"""
import math

import numpy as np
import torch

own = False

DV = 128
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
DEV = "cuda"


def _pad16(n):
    return (n + 15) // 16 * 16


def kv_bytes(kv, d):
    """Bytes of a cached row of d values."""
    return {"bf16": 2 * d, "fp8": d, "fp4": _pad16(d // 2 + d // 16)}[kv]


def bounds_bytes(d):
    """Bytes of a block's bounds: d upper codes, d lower ones, their exponent, padding."""
    return _pad16(2 * d + 1)


def listed():
    base = dict(kv="bf16", batch=1, len_min=512, len_max=512, new=1, mixed=False, hq=16, hkv=2, dqk=192,
                page=128, len_seed=1)

    def mrope(name, **kw):
        return {**base, **dict(name=name, op="mrope", pairs=False, axes=3, layout="sections", given=True,
                               rot=64, rot_off=0), **kw}

    def bounds(name, **kw):
        return {**base, **dict(name=name, op="bounds", block=64, whole=False), **kw}

    def select(name, **kw):
        return {**base, **dict(name=name, op="select", block=64, take=16, first=1, last=2), **kw}

    def sparse(name, **kw):
        return {**base, **dict(name=name, op="sparse", block=64, take=16, first=1, last=2, sinks=False), **kw}

    return [
        # the decode step behind a video prompt: one text token a request, all axes alike
        mrope("mrope_decode", kv="fp8", batch=33, len_min=1024, len_max=4096, given=False),
        # image patches of a batch of short prompts, neighbours paired, the rotated part last
        mrope("mrope_image", batch=7, len_min=900, len_max=2500, new=333, page=64, pairs=True,
              layout="interleaved", rot_off=128),
        # a chunk of video frames into an 8-bit cache, 64 query heads
        mrope("mrope_video", kv="fp8", len_min=30096, len_max=30096, new=4096, hq=64, hkv=4,
              layout="interleaved"),
        # draft tokens: one request in eight completes a block
        bounds("bounds_verify", kv="fp8", batch=64, len_min=2000, len_max=9000, new=8),
        # a 4-bit cache that came without its bounds: all blocks of all requests
        bounds("bounds_rebuild", kv="fp4", batch=16, len_min=1024, len_max=32767, hkv=4, whole=True),
        # a serving batch of ragged long requests, one token each
        select("select_decode", batch=32, len_min=1024, len_max=32767),
        # one very long request: the blocks are many and the query rows few
        select("select_long", len_min=524288, len_max=524288, hq=64, hkv=4, block=32, take=64),
        # a prompt's later chunk: every token chooses among the blocks before it
        select("select_prefill", len_min=30096, len_max=30096, new=4096, hq=64, hkv=4),
        # the same serving batch, attending to 16 blocks of 64 keys
        sparse("sparse_decode", batch=32, len_min=1024, len_max=32767),
        # speculative decoding over an 8-bit cache, sinks
        sparse("sparse_verify", kv="fp8", batch=4, len_min=46008, len_max=46008, new=8, sinks=True),
        # a ragged chunk over a 4-bit cache, blocks of 128
        sparse("sparse_chunk_fp4", kv="fp4", batch=3, len_min=5000, len_max=20000, new=777, hq=32, hkv=8,
               block=128, take=12),
        # a prompt's later chunk over a bf16 cache
        sparse("sparse_prefill", len_min=30096, len_max=30096, new=4096, hq=64, hkv=4),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    """One more case of the same ranges."""
    hq, hkv = rng.choice([(8, 1), (16, 2), (64, 4), (12, 3), (32, 8), (4, 4), (40, 2)])
    dqk = rng.choice([192, 192, 128])
    kv = rng.choice(["bf16", "fp8", "fp4"])
    op = rng.choice(["mrope", "bounds", "select", "select", "sparse", "sparse"])
    c = dict(op=op, kv=kv, hq=hq, hkv=hkv, dqk=dqk, len_seed=rng.randrange(1 << 20))
    if op == "mrope":
        rot = 16 * rng.randint(1, dqk // 16)
        batch = _log_int(rng, 1, 64)
        new = _log_int(rng, 1, max(1, min(1500, 180_000_000 // ((4 * dqk * hq + 6 * hkv * (dqk + DV)) * batch))))
        hi = new + _log_int(rng, 1, 3000)
        return dict(batch=batch, len_min=max(new, hi // 2), len_max=hi, new=new, mixed=False,
                    page=rng.choice([1, 3, 16, 32, 64, 128]), pairs=rng.random() < 0.5, axes=rng.choice([2, 3, 3, 4]),
                    layout=rng.choice(["sections", "interleaved"]), given=rng.random() < 0.7, rot=rot,
                    rot_off=8 * rng.randint(0, (dqk - rot) // 8), **c)
    block = rng.choice([16, 32, 64, 64, 128])
    c.update(block=block, page=block * rng.choice([1, 1, 2, 3, 4]))
    kind = rng.choice(["decode", "decode", "verify", "chunk"])
    new = {"decode": 1, "verify": rng.randint(2, 16), "chunk": _log_int(rng, 33, 900)}[kind]
    batch = 1 if kind == "chunk" else _log_int(rng, 1, 48)
    top = max(new + 1, min(800_000 // hkv // batch, 24_000 if kind == "chunk" else 60_000))
    hi = max(new, _log_int(rng, min(new + 1, top), top))
    c.update(batch=batch, new=new, len_min=max(new, hi // rng.choice([1, 2, 30])), len_max=hi,
             mixed=kind == "verify" and rng.random() < 0.5)
    if op == "bounds":
        if hi < 2 * block:                      # some block is whole
            c.update(len_min=2 * block, len_max=2 * block + hi)
        c["whole"] = rng.random() < 0.3
        L, n = _lengths(c)
        return dict(c, whole=c["whole"] or not (L // block > (L - n) // block).any())
    last = rng.choice([1, 2, 3])
    if hi < 16 * block:                         # there is something to choose from
        c.update(len_min=16 * block, len_max=16 * block + hi)
    blocks = c["len_max"] // block
    c.update(first=rng.choice([0, 1, 2]), last=last, take=max(last + 3, min(_log_int(rng, 4, 40), blocks // 2)))
    return dict(sinks=rng.random() < 0.5, **c) if op == "sparse" else c


def _lengths(case):
    """Requests' lengths and new tokens, from the case alone."""
    rng = np.random.default_rng(case["len_seed"])
    L = rng.integers(case["len_min"], case["len_max"] + 1, size=case["batch"]).astype(np.int64)
    n = np.full(case["batch"], case["new"], np.int64)
    if case.get("mixed"):
        n[::2] = 1
    return L, n


def _completed(case, L, n):
    """(first, end) of the blocks that the operator `bounds` writes, per request."""
    end = L // case["block"]
    return (np.zeros_like(L) if case["whole"] else (L - n) // case["block"]), end


def _pair_axis(case):
    """Which axis turns each pair of dimensions."""
    half, A = case["rot"] // 2, case["axes"]
    if case["layout"] == "interleaved":
        return [i % A for i in range(half)]
    cuts = [half * (2 * k + 1) // (2 * A) if k < A else half for k in range(A + 1)]
    cuts[0] = 0
    return [max(k for k in range(A) if cuts[k] <= i) for i in range(half)]


def _lists(score, own_block, case, xp):
    """Block lists of tokens, from a score per (token, head, block): the first and last blocks and the
    highest scores up to `take`, ascending, -1 behind.  xp: torch; own_block [T] int64."""
    C = score.shape[-1]
    c = xp.arange(C, device=score.device)
    ob = own_block[:, None, None]
    s = xp.where((c < case["first"]) | (c > ob - case["last"]), xp.full_like(score, math.inf),
                 score.clamp(max=3e38))
    s = xp.where(c <= ob, s, xp.full_like(s, -math.inf))
    take = min(case["take"], C)
    order = xp.sort(s, dim=-1, descending=True, stable=True).indices[..., :take]
    order = xp.where(order <= ob, order, xp.full_like(order, C))
    order = xp.sort(order, dim=-1).values
    out = xp.full((*score.shape[:2], case["take"]), -1, dtype=xp.int32, device=score.device)
    out[..., :take] = xp.where(order < C, order, xp.full_like(order, -1)).int()
    return out


def _drawn_scores(g, tokens, heads, C, device):
    """Scores whose high ones stay for a stretch of tokens, as those of neighbouring queries do."""
    runs = torch.randn((tokens + 15) // 16, heads, C, generator=g, device=device)
    return runs.repeat_interleave(16, 0)[:tokens] + 0.5 * torch.randn(tokens, heads, C, generator=g, device=device)


def _union_blocks(case, L, n):
    """Blocks that one KV head's tokens of a request attend to, all together (of lists drawn as
    prepare draws them)."""
    if n == 1:
        return min(case["take"], (L - 1) // case["block"] + 1)
    g = torch.Generator()
    g.manual_seed(1)
    C = (L - 1) // case["block"] + 1
    own_block = torch.arange(L - n, L) // case["block"]
    return int(_lists(_drawn_scores(g, n, 1, C, "cpu"), own_block, case, torch).unique().ge(0).sum())


def work(case):
    L, n = _lengths(case)
    T, hq, hkv, dqk, kv = int(n.sum()), case["hq"], case["hkv"], case["dqk"], case["kv"]
    index = 4.0 * (2 * len(L) + 1)
    per = {"bf16": 2.0, "fp8": 1.0, "fp4": 0.5 + 1 / 16}[kv]
    if case["op"] == "mrope":
        b = T * hkv * (dqk + DV) * (2.0 + per)            # the cache's rows, written
        b += T * hkv * (dqk + DV) * (0.0 if kv == "bf16" else per + 2.0)   # and read back
        b += T * (2.0 * hq * 2 * dqk + 4.0 * case["rot"] + (4.0 * case["axes"] if case["given"] else 0.0))
        return {"bytes": b + index + 4.0 * T, "flops": 3.0 * T * (hq + hkv) * case["rot"]}
    Bs = case["block"]
    if case["op"] == "bounds":
        lo, hi = _completed(case, L, n)
        blocks = float((hi - lo).sum()) * hkv
        return {"bytes": blocks * (Bs * dqk * per + 2 * dqk + 1 + 2 * dqk + 1 + 4 * dqk) + index,
                "flops": blocks * 2 * Bs * dqk}
    i = np.concatenate([np.arange(a - b, a) for a, b in zip(L, n)])
    own_block = i // Bs
    if case["op"] == "select":
        mid = np.maximum(0, own_block - case["last"] + 1 - case["first"])
        last = np.array([max(0, int((a - 1) // Bs) - case["last"] + 1 - case["first"]) for a in L])
        return {"bytes": float(last.sum()) * hkv * (2 * dqk + 1) + T * (2.0 * hq * dqk + 4.0 * hkv * case["take"])
                + index + 4.0 * float(last.sum()), "flops": 2.0 * dqk * hq * float(mid.sum())}
    keys = sum(_union_blocks(case, a, b) for a, b in zip(L.tolist(), n.tolist())) * Bs
    keys -= float(((own_block[np.cumsum(n) - 1] + 1) * Bs - L).sum())          # the last block ends at L
    taken = np.minimum(case["take"], own_block + 1)
    visible = (taken - 1) * Bs + i % Bs + 1
    return {"bytes": keys * hkv * (dqk + DV) * per + T * (hq * (2.0 * dqk + 2.0 * DV + 4) + 4.0 * hkv * case["take"])
            + index + 4.0 * keys / Bs, "flops": 2.0 * float(visible.sum()) * hq * (dqk + DV)}


# --------------------------------------------------------------------------- cached rows, plain

def _quantise(x, scale):
    """fp32 [..., d] -> uint8 rows of the 4-bit cache."""
    d = x.shape[-1]
    y = (x / scale).unflatten(-1, (d // 16, 16))
    s = (y.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    sf = s.float().unsqueeze(-1)
    a = torch.where(sf > 0, y.abs() / sf, torch.zeros_like(y))
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5)
            + (a > 5.0))
    code = (code + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2)
    packed = code[..., 0::2] + 16 * code[..., 1::2]
    pad = kv_bytes("fp4", d) - d // 2 - d // 16
    zeros = torch.zeros(*x.shape[:-1], pad, dtype=torch.uint8, device=x.device)
    return torch.cat([packed, s.view(torch.uint8), zeros], -1)


def _store(x, scale, kv):
    """fp32 values as cached rows."""
    if kv == "bf16":
        return x.bfloat16()
    if kv == "fp8":
        return (x / scale).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    return _quantise(x, scale)


def _values(rows, d, kv, lut):
    """Cached rows -> fp32 [..., d], without the tensor's scale; lut: E2M1's 16 values."""
    if kv == "bf16":
        return rows.float()
    if kv == "fp8":
        return rows.view(torch.float8_e4m3fn).float()
    b = rows[..., : d // 2]
    v = lut[torch.stack([b & 15, b >> 4], -1).flatten(-2).int()]
    s = rows[..., d // 2: d // 2 + d // 16].contiguous().view(torch.float8_e4m3fn).float()
    return (v.unflatten(-1, (d // 16, 16)) * s.unsqueeze(-1)).flatten(-2)


def _exponent(amax):
    """The least e with amax <= 127 * 2^e, within [-126, 121]; 0 for amax = 0."""
    m, x = torch.frexp(amax)
    e = (x - 7 + (m > 127 / 128).int()).clamp(-126, 121)
    return torch.where(amax > 0, e, torch.zeros_like(e))


def _record(hi, lo):
    """fp32 upper and lower bounds [..., d] -> a block's record: codes rounded outwards, exponent."""
    d = hi.shape[-1]
    e = _exponent(torch.maximum(hi.abs(), lo.abs()).amax(-1))
    unit = torch.ldexp(torch.ones_like(hi[..., 0]), -e).unsqueeze(-1)
    rec = torch.zeros(*hi.shape[:-1], bounds_bytes(d), dtype=torch.int8, device=hi.device)
    rec[..., :d] = (hi * unit).ceil().to(torch.int8)
    rec[..., d:2 * d] = (lo * unit).floor().to(torch.int8)
    rec[..., 2 * d] = e.to(torch.int8)
    return rec.view(torch.uint8)


# --------------------------------------------------------------------------- inputs

def _pool(g, slots, hkv, d, scale, kv, std):
    """Rows of a pool of `slots` slots, filled as earlier appends left them."""
    x = torch.randn(slots, hkv, d, generator=g, device=DEV) * std
    x += torch.randn(1, hkv, d, generator=g, device=DEV) * (0.5 * std)      # keys have a mean
    return _store(x, scale, kv)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    L, n = _lengths(case)
    op, kv = case["op"], case["kv"]
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
    lens = torch.tensor(L, dtype=torch.int32, device=DEV)
    qo = torch.tensor(np.concatenate([[0], np.cumsum(n)]), dtype=torch.int32, device=DEV)
    top = {"bf16": None, "fp8": 448.0, "fp4": 6.0 * 448.0}[kv]
    ks, vs = (1.0, 1.0) if top is None else (float(np.float32(5.4371 / top)), float(np.float32(6.0193 / top)))
    pos = torch.tensor(np.concatenate([np.arange(a - b, a) for a, b in zip(L, n)]), device=DEV)
    s = dict(case=case, L=L, n=n, T=T, page_table=table, qo=qo, lens=lens, k_scale=ks, v_scale=vs,
             num_pages=num_pages, req=torch.tensor(np.repeat(np.arange(B), n), device=DEV), pos=pos,
             lut=torch.tensor(E2M1 + tuple(-v for v in E2M1), device=DEV))
    if op != "bounds":
        # queries: what neighbouring tokens and the heads of a group share, and their own part
        q = torch.randn(T, hq, dqk, generator=g, device=DEV)
        runs = torch.randn((T + 15) // 16, hkv, 1, dqk, generator=g, device=DEV).repeat_interleave(16, 0)[:T]
        s["q"] = (q.view(T, hkv, hq // hkv, dqk) + runs).view(T, hq, dqk).bfloat16()
    if op != "select":
        s["k_cache"] = _pool(g, num_pages * P, hkv, dqk, ks, kv, 0.8).view(num_pages, P, hkv, -1)
    if op in ("mrope", "sparse"):
        s["v_cache"] = _pool(g, num_pages * P, hkv, DV, vs, kv, 1.0).view(num_pages, P, hkv, -1)
    if op == "mrope":
        s["k_new"] = (torch.randn(T, hkv, dqk, generator=g, device=DEV) * 0.8).bfloat16()
        s["v_new"] = torch.randn(T, hkv, DV, generator=g, device=DEV).bfloat16()
        half, A = case["rot"] // 2, case["axes"]
        inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=DEV) / half)
        ang = torch.arange(int(L.max()) + 1, dtype=torch.float64, device=DEV)[:, None] * inv
        s["cos_sin"] = torch.cat([ang.cos(), ang.sin()], -1).float().contiguous()
        s["pair_axis"] = _pair_axis(case)
        s["axis_of"] = torch.tensor(s["pair_axis"], device=DEV)
        if case["given"]:
            # frames of 24 x 36 patches in raster order behind what came before
            start = torch.tensor(L - n, device=DEV)[s["req"]]
            t = pos - start
            axes = [start + t // 864, start + t % 864 // 36, start + t % 36, start][:A]
            s["positions"] = torch.minimum(torch.stack(axes), pos).int().contiguous()
        else:
            # text behind images: positions run behind the tokens' count
            back = torch.rand(B, generator=g, device=DEV) * torch.tensor(L - n, device=DEV)
            s["delta"] = -back.int()
    if op in ("sparse", "select"):
        Bs = case["block"]
        C = int((L.max() - 1) // Bs) + 1
        s["own_block"] = pos // Bs
    if op == "sparse":
        s["block_idx"] = _lists(_drawn_scores(g, T, hkv, C, DEV), s["own_block"], case, torch).contiguous()
        s["sinks"] = torch.randn(hq, generator=g, device=DEV) if case["sinks"] else None
        s["scale"] = 1.0 / math.sqrt(dqk)
        # slots behind a request's last key, and pages nobody owns, were never written
        key = torch.arange(stride * P, device=DEV)
        slot = table.long()[:, key // P] * P + key % P
        used = torch.zeros(num_pages * P, dtype=torch.bool, device=DEV)
        used[slot[key < lens[:, None]]] = True
        for name in ("k_cache", "v_cache"):
            s[name].view(num_pages * P, -1)[~used] = float("nan") if kv == "bf16" else 0xFF
    if op in ("select", "bounds"):
        slots = num_pages * (P // case["block"])
        x = torch.randn(slots, hkv, dqk, generator=g, device=DEV) * 0.7
        r = 1.0 + 0.6 * torch.rand(slots, hkv, dqk, generator=g, device=DEV)
        s["bounds"] = _record(x + r, x - r).view(num_pages, P // case["block"], hkv, -1)
    if op == "bounds":
        lo, hi = _completed(case, L, n)
        s["lo"], s["hi"] = torch.tensor(lo, device=DEV), torch.tensor(hi, device=DEV)
        s["blocks"] = int((hi - lo).sum())
        rows = L if case["whole"] else n
        s["rows"] = int(rows.sum())
        s["kv_indptr"] = torch.tensor(np.concatenate([[0], np.cumsum(rows)]), dtype=torch.int32, device=DEV)
        s["block_indptr"] = torch.tensor(np.concatenate([[0], np.cumsum(hi - lo)]), dtype=torch.int32, device=DEV)
    if own:
        from asymmetric_kv_paged_gb300 import binding as B_
        kinds = {"bf16": B_.ATTN_KV_BF16, "fp8": B_.ATTN_KV_FP8_E4M3, "fp4": B_.ATTN_KV_FP4_E2M1}
        prob, keep = B_.make_problem(
            batch=B, num_q_heads=hq, num_kv_heads=hkv, page_size=P, num_pages=num_pages,
            page_table_stride=stride, kv_dtype=kinds[kv], window=0, has_sinks=case.get("sinks", False),
            qo_indptr=np.concatenate([[0], np.cumsum(n)]), seq_lens=L, head_dim_qk=dqk)
        s["plan"] = B_.attn_plan(prob, torch.cuda.current_device(), keep)
        bf = dict(dtype=torch.bfloat16, device=DEV)
        if op == "mrope":
            s["k_read"], s["v_read"] = torch.empty(T, hkv, dqk, **bf), torch.empty(T, hkv, DV, **bf)
            s["q_out"] = torch.empty(T, hq, dqk, **bf)
            s["mrope"] = B_.make_mrope(s["cos_sin"], case["rot"], s["pair_axis"], positions=s.get("positions"),
                                       position_delta=s.get("delta"), rot_offset=case["rot_off"],
                                       interleaved=case["pairs"])
        elif op == "bounds":
            s["read"] = torch.empty(s["blocks"], hkv, 2, dqk, **bf)
        else:
            s["sparse"] = B_.make_sparse(case["block"], case["take"], case["first"], case["last"])
            if op == "select":
                s["picked"] = torch.empty(T, hkv, case["take"], dtype=torch.int32, device=DEV)
            else:
                s["out"] = torch.empty(T, hq, DV, **bf)
                s["lse"] = torch.empty(T, hq, dtype=torch.float32, device=DEV)
    return s


# --------------------------------------------------------------------------- one pass

def _rotate(x, cos, sin, case):
    """x fp32 [T, H, d]; cos, sin [T, 1, rot / 2]."""
    rot, off = case["rot"], case["rot_off"]
    part = x[..., off: off + rot]
    if case["pairs"]:
        x1, x2 = part[..., 0::2], part[..., 1::2]
        turned = torch.stack([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1).flatten(-2)
    else:
        x1, x2 = part[..., : rot // 2], part[..., rot // 2:]
        turned = torch.cat([x1 * cos - x2 * sin, x2 * cos + x1 * sin], -1)
    return torch.cat([x[..., :off], turned, x[..., off + rot:]], -1)


def _angle_rows(s):
    """The table's row for every (token, pair)."""
    if s["case"]["given"]:
        return s["positions"].long()[s["axis_of"]].T
    return (s["pos"] + s["delta"].long()[s["req"]])[:, None].expand(-1, s["case"]["rot"] // 2)


def _mrope_plain(s):
    c = s["case"]
    P, kv, half = c["page"], c["kv"], c["rot"] // 2
    rows, i = _angle_rows(s), torch.arange(half, device=DEV)
    cos, sin = s["cos_sin"][rows, i][:, None], s["cos_sin"][rows, half + i][:, None]
    k = _rotate(s["k_new"].float(), cos, sin, c)
    out = {"q": _rotate(s["q"].float(), cos, sin, c).bfloat16()}
    slot = s["page_table"].long()[s["req"], s["pos"] // P] * P + s["pos"] % P
    kc, vc = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    kc[slot], vc[slot] = _store(k, s["k_scale"], kv), _store(s["v_new"].float(), s["v_scale"], kv)
    if kv == "bf16":
        return {**out, "k": s["k_cache"], "v": s["v_cache"]}
    out["k"] = (_values(kc[slot], c["dqk"], kv, s["lut"]) * s["k_scale"]).bfloat16()
    out["v"] = (_values(vc[slot], DV, kv, s["lut"]) * s["v_scale"]).bfloat16()
    return out


def _bounds_plain(s):
    c = s["case"]
    P, Bs = c["page"], c["block"]
    b = torch.repeat_interleave(torch.arange(c["batch"], device=DEV), s["hi"] - s["lo"])
    blk = torch.arange(s["blocks"], device=DEV) - s["block_indptr"].long()[b] + s["lo"][b]
    out = torch.empty(s["blocks"], c["hkv"], 2, c["dqk"], dtype=torch.bfloat16, device=DEV)
    step = max(1, 2 ** 28 // (Bs * c["hkv"] * c["dqk"]))
    for i in range(0, s["blocks"], step):
        bb, cc = b[i:i + step], blk[i:i + step]
        page = s["page_table"].long()[bb, cc * Bs // P]
        slot = (page * P + cc * Bs % P)[:, None] + torch.arange(Bs, device=DEV)
        K = _values(s["k_cache"].flatten(0, 1)[slot], c["dqk"], c["kv"], s["lut"])
        rec = _record(K.amax(1), K.amin(1))
        s["bounds"][page, cc * Bs % P // Bs] = rec
        codes = rec.view(torch.int8).float()
        unit = torch.ldexp(torch.ones_like(codes[..., 0]), codes[..., 2 * c["dqk"]].int())[..., None, None]
        out[i:i + step] = (codes[..., : 2 * c["dqk"]].unflatten(-1, (2, c["dqk"])) * unit).bfloat16()
    return {"bounds": out}


def _select_plain(s):
    c = s["case"]
    B, P, Bs, hkv, dqk = c["batch"], c["page"], c["block"], c["hkv"], c["dqk"]
    G = c["hq"] // hkv
    q = s["q"].float().view(s["T"], hkv, G, dqk)
    e = _exponent(q.abs().amax(-1))                                           # [T, hkv, G]
    q = (q * torch.ldexp(torch.ones_like(q[..., 0]), -e)[..., None]).round()
    f = torch.ldexp(torch.ones_like(q[..., 0]), e - e.amax(-1, keepdim=True))
    C = int((s["L"].max() - 1) // Bs) + 1
    score = torch.zeros(s["T"], hkv, C, device=DEV)
    t0 = 0
    for b, (L, n) in enumerate(zip(s["L"].tolist(), s["n"].tolist())):
        nb = (L - 1) // Bs + 1
        blk = torch.arange(nb, device=DEV)
        page = s["page_table"][b].long()[blk * Bs // P]
        rec = s["bounds"][page, blk * Bs % P // Bs].view(torch.int8).float()       # [nb, hkv, row]
        unit = torch.ldexp(torch.ones_like(rec[..., 0]), rec[..., 2 * dqk].int()).T  # [hkv, nb]
        hi, lo = rec[..., :dqk].permute(1, 2, 0), rec[..., dqk:2 * dqk].permute(1, 2, 0)
        for i in range(0, n, 1024):
            j = slice(t0 + i, t0 + min(n, i + 1024))
            qq = q[j].permute(1, 0, 2, 3).flatten(1, 2)                       # [hkv, t * G, d]
            dot = qq.clamp(min=0) @ hi + qq.clamp(max=0) @ lo
            dot = dot.unflatten(1, (-1, G)) * f[j].permute(1, 0, 2)[..., None]
            score[j, :, :nb] = (dot.amax(2) * unit[:, None]).permute(1, 0, 2)
        t0 += n
    return {"blocks": _lists(score, s["own_block"], c, torch)}


def _sparse_plain(s):
    c = s["case"]
    P, Bs, hkv, dqk, kv, S = c["page"], c["block"], c["hkv"], c["dqk"], c["kv"], c["take"]
    G, T = c["hq"] // hkv, s["T"]
    out = torch.empty(T, c["hq"], DV, dtype=torch.bfloat16, device=DEV)
    lse = torch.empty(T, c["hq"], device=DEV)
    head = torch.arange(hkv, device=DEV)[:, None]
    kc, vc = s["k_cache"].flatten(0, 1), s["v_cache"].flatten(0, 1)
    step = max(1, 2 ** 28 // (hkv * S * Bs * dqk))
    for i in range(0, T, step):
        idx = s["block_idx"][i:i + step].long()                               # [t, hkv, S]
        t = idx.shape[0]
        key = (idx[..., None] * Bs + torch.arange(Bs, device=DEV)).flatten(-2)
        see = (key >= 0) & (key <= s["pos"][i:i + step, None, None])
        key = torch.where(see, key, torch.zeros_like(key))
        page = s["page_table"].long()[s["req"][i:i + step, None, None], key // P]
        slot = page * P + key % P
        K = _values(kc[slot, head], dqk, kv, s["lut"]) * s["k_scale"]         # [t, hkv, keys, d]
        q = s["q"][i:i + step].float().view(t, hkv, G, dqk)
        S_ = (q @ K.transpose(-1, -2)) * s["scale"]
        del K
        S_.masked_fill_(~see[:, :, None], -math.inf)
        m = S_.amax(-1, keepdim=True)
        if s["sinks"] is not None:
            sink = s["sinks"].view(hkv, G, 1)
            m = torch.maximum(m, sink)
        p = S_.sub_(m).exp_()
        z = p.sum(-1, keepdim=True)
        if s["sinks"] is not None:
            z = z + (sink - m).exp()
        V = _values(vc[slot, head], DV, kv, s["lut"]) * s["v_scale"]
        out[i:i + step] = ((p @ V) / z).flatten(1, 2).bfloat16()
        lse[i:i + step] = (m + z.log()).flatten(1, 3)
    return {"out": out, "lse": lse}


def run(s):
    c = s["case"]
    op = c["op"]
    if not own:
        return {"mrope": _mrope_plain, "bounds": _bounds_plain, "select": _select_plain, "sparse": _sparse_plain}[op](s)
    from asymmetric_kv_paged_gb300 import binding as B_
    if op == "mrope":
        B_.attn_append_kv_mrope(s["plan"], s["mrope"], s["q"], s["k_new"], s["v_new"], s["q_out"], s["k_cache"],
                                s["v_cache"], s["page_table"], s["lens"], s["qo"], s["k_scale"], s["v_scale"])
        if c["kv"] == "bf16":
            return {"q": s["q_out"], "k": s["k_cache"], "v": s["v_cache"]}
        B_.attn_read_kv(s["plan"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"], s["qo"], s["k_read"],
                        s["v_read"], s["k_scale"], s["v_scale"])
        return {"q": s["q_out"], "k": s["k_read"], "v": s["v_read"]}
    if op == "bounds":
        B_.attn_update_bounds(s["plan"], c["block"], s["k_cache"], s["bounds"], s["page_table"], s["lens"],
                              s["kv_indptr"], s["rows"])
        B_.attn_read_bounds(s["plan"], c["block"], s["bounds"], s["page_table"], s["lens"], s["block_indptr"], s["read"])
        return {"bounds": s["read"]}
    if op == "select":
        B_.attn_select_blocks(s["plan"], s["sparse"], s["q"], s["bounds"], s["page_table"], s["lens"], s["qo"],
                              s["picked"])
        return {"blocks": s["picked"]}
    B_.attn_run_sparse(s["plan"], s["sparse"], s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["lens"],
                       s["qo"], s["block_idx"], s["sinks"], s["scale"], s["k_scale"], s["v_scale"], s["out"], s["lse"])
    return {"out": s["out"], "lse": s["lse"]}


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


def _decode64(rows, d, kv):
    """Cached rows from the formats' bit fields, in 64 bits."""
    if kv == "bf16":
        return rows.double()
    t8 = _e4m3_table()
    r = rows.long()
    if kv == "fp8":
        v = t8[(r % 128).clamp(max=126)]
        return torch.where(r >= 128, -v, v)
    code = torch.stack([r[..., : d // 2] % 16, r[..., : d // 2] // 16], -1).flatten(-2)
    e, m = code // 2 % 4, code % 2
    mag = torch.where(e == 0, m * 0.5, (1 + m * 0.5) * torch.exp2((e - 1).double()))
    val = torch.where(code >= 8, -mag, mag)
    return val * t8[r[..., d // 2: d // 2 + d // 16].clamp(max=126)].repeat_interleave(16, -1)


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


def _mrope64(s):
    c = s["case"]
    half, off = c["rot"] // 2, c["rot_off"]
    at = torch.arange(half, device=DEV)
    w = torch.empty(s["T"], 1, half, dtype=torch.complex128, device=DEV)
    for i, axis in enumerate(_pair_axis(c)):
        row = s["positions"][axis].long() if c["given"] else s["pos"] + s["delta"].long()[s["req"]]
        w[:, 0, i] = torch.complex(s["cos_sin"][row, i].double(), s["cos_sin"][row, half + i].double())
    i1, i2 = (off + 2 * at, off + 2 * at + 1) if c["pairs"] else (off + at, off + half + at)

    def turn(x):
        y = x.clone()
        z = torch.complex(x[..., i1], x[..., i2]) * w
        y[..., i1], y[..., i2] = z.real, z.imag
        return y

    k, v = turn(s["k_new"].double()), s["v_new"].double()
    out = {"q": turn(s["q"].double())}
    if c["kv"] == "bf16":
        P = c["page"]
        slot = s["page_table"].long()[s["req"], s["pos"] // P] * P + s["pos"] % P
        kc, vc = s["k_cache"].double(), s["v_cache"].double()
        kc.flatten(0, 1)[slot], vc.flatten(0, 1)[slot] = k, v
        return {**out, "k": kc, "v": vc}
    return {**out, "k": _round64(k, s["k_scale"], c["kv"]), "v": _round64(v, s["v_scale"], c["kv"])}


def _unit64(amax):
    """The smallest power of two that amax / 127 does not exceed."""
    e = torch.ceil(torch.log2(torch.where(amax > 0, amax, torch.full_like(amax, 127.0)) / 127))
    e = e + (torch.exp2(e) * 127 < amax).double() - (torch.exp2(e - 1) * 127 >= amax).double() * (amax > 0)
    return torch.exp2(e.clamp(-126, 121))


def _bounds64(s):
    c = s["case"]
    P, Bs = c["page"], c["block"]
    out, kc = [], s["k_cache"].flatten(0, 1)
    lo, hi = _completed(c, s["L"], s["n"])
    for b in range(c["batch"]):
        for first in range(int(lo[b]), int(hi[b]), 256):
            j = torch.arange(first * Bs, min(first + 256, int(hi[b])) * Bs, device=DEV)
            K = _decode64(kc[s["page_table"][b].long()[j // P] * P + j % P], c["dqk"], c["kv"])
            K = K.unflatten(0, (-1, Bs))
            top, bot = K.max(1).values, K.min(1).values
            u = _unit64(K.abs().amax((1, 3)))[..., None]
            out.append(torch.stack([torch.ceil(top / u) * u, torch.floor(bot / u) * u], 2))
    if not out:
        return {"bounds": torch.zeros(0, c["hkv"], 2, c["dqk"], dtype=torch.float64, device=DEV)}
    return {"bounds": torch.cat(out)}


def _select64(s):
    c = s["case"]
    P, Bs, hkv, dqk, S = c["page"], c["block"], c["hkv"], c["dqk"], c["take"]
    G = c["hq"] // hkv
    if work(c)["flops"] > 1e11:
        return {"blocks": None}
    out = torch.full((s["T"], hkv, S), -1, dtype=torch.int32, device=DEV)
    t0 = 0
    for b, (L, n) in enumerate(zip(s["L"].tolist(), s["n"].tolist())):
        blk = torch.arange((L - 1) // Bs + 1, device=DEV)
        rec = s["bounds"][s["page_table"][b].long()[blk * Bs // P], blk * Bs % P // Bs].view(torch.int8).double()
        u = torch.exp2(rec[..., 2 * dqk])[..., None]
        hi, lo = rec[..., :dqk] * u, rec[..., dqk:2 * dqk] * u                # [nb, hkv, d]
        step = max(1, 2 ** 27 // (len(blk) * hkv * dqk))
        for i in range(0, n, step):
            q = s["q"][t0 + i:t0 + min(n, i + step)].double().unflatten(1, (hkv, G))
            uq = _unit64(q.abs().amax(-1))[..., None]
            q = torch.round(q / uq) * uq
            best = None
            for h in range(G):
                x = q[:, None, :, h]                                          # [t, 1, hkv, d]
                v = torch.maximum(x * hi, x * lo).sum(-1)
                best = v if best is None else torch.maximum(best, v)          # [t, nb, hkv]
            for k in range(q.shape[0]):
                nb = (L - n + i + k) // Bs + 1
                v = best[k, :nb].clone()
                forced = (blk[:nb] < c["first"]) | (blk[:nb] >= nb - c["last"])
                v[forced] = math.inf
                pick = torch.argsort(-v, dim=0, stable=True)[:S].sort(0).values
                out[t0 + i + k, :, :pick.shape[0]] = pick.T.int()
        t0 += n
    return {"blocks": out}


def _sparse64(s):
    c = s["case"]
    P, Bs, hkv, dqk = c["page"], c["block"], c["hkv"], c["dqk"]
    G = c["hq"] // hkv
    out = torch.zeros(s["T"], c["hq"], DV, dtype=torch.float64, device=DEV)
    lse = torch.zeros(s["T"], c["hq"], dtype=torch.float64, device=DEV)
    within = torch.arange(Bs, device=DEV)
    t0 = 0
    for b, (L, n) in enumerate(zip(s["L"].tolist(), s["n"].tolist())):
        j = torch.arange(L, device=DEV)
        slot = s["page_table"][b].long()[j // P] * P + j % P
        for g in range(hkv):
            K = _decode64(s["k_cache"].flatten(0, 1)[slot, g], dqk, c["kv"]) * s["k_scale"]
            V = _decode64(s["v_cache"].flatten(0, 1)[slot, g], DV, c["kv"]) * s["v_scale"]
            for i in range(0, n, 128):
                t = torch.arange(t0 + i, t0 + min(n, i + 128), device=DEV)
                key = (s["block_idx"][t, g].long()[..., None] * Bs + within).flatten(1)   # [t, keys]
                bad = (key < 0) | (key > s["pos"][t][:, None])
                key = key.clamp(0, L - 1)
                q = s["q"][t, g * G:(g + 1) * G].double()
                S = torch.einsum("thd,tkd->thk", q, K[key]) * s["scale"]
                S = torch.where(bad[:, None], -math.inf, S)
                Z = torch.logsumexp(S, -1)
                if s["sinks"] is not None:
                    Z = torch.logaddexp(Z, s["sinks"][g * G:(g + 1) * G].double())
                out[t, g * G:(g + 1) * G] = torch.einsum("thk,tkd->thd", torch.exp(S - Z[..., None]), V[key])
                lse[t, g * G:(g + 1) * G] = Z
        t0 += n
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"mrope": _mrope64, "bounds": _bounds64, "select": _select64, "sparse": _sparse64}[case["op"]](s)
