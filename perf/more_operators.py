"""The operators of a paged cache held in 4 bits, and the read-back of cached rows, as cases that can be timed and compared.

A row of head_dim values is held as e2m1 codes (two a byte, the even dim in the low bits) under one e4m3 scale for every
16 dims, times a power of two for the layer's K and one for its V:

    value = e2m1(code) * e4m3(block scale) * 2^exp

Three operators that a serving loop over such a cache runs:
  store   new K / V rows quantised into their slots as they are written, and the same slots read back, as the attention
          of the chunk they belong to wants them (what decode will see, not what was written)
  read    the rows of cached tokens, by slot, as bf16: from a 4-bit, an e4m3 or a bf16 cache
  decode  attention of each request's newest tokens over its 4-bit cache, global or sliding-window

With `own` false, run() computes an operator in its plain form from elementary torch operations; with `own` true it
makes the calls a user makes of the framework.
"""
import math

import torch

own = False

# query heads, KV heads, head_dim of the layer kinds served here
LAYERS = ((16, 4, 512), (8, 2, 512), (16, 8, 256), (32, 4, 256), (24, 4, 512))
BLOCK = 16  # dims under one scale
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


def listed():
    return [
        # one decode step's rows, where latency counts
        {"name": "store decode t64", "op": "store", "tokens": 64, "kv_heads": 4, "dim": 512, "page": 16,
         "kv_shared": False, "fused": True, "padding": 0.0, "k_exp": 0, "v_exp": -4},
        # a prompt's rows out of a fused QKV projection
        {"name": "store prompt t16384", "op": "store", "tokens": 16384, "kv_heads": 4, "dim": 512, "page": 16,
         "kv_shared": False, "fused": True, "padding": 0.0, "k_exp": 0, "v_exp": -4},
        # ragged chunks padded to a fixed count, the other layer kind
        {"name": "store ragged t20011", "op": "store", "tokens": 20011, "kv_heads": 8, "dim": 256, "page": 32,
         "kv_shared": False, "fused": False, "padding": 0.1, "k_exp": 1, "v_exp": -2},
        # the few cached rows in front of a short chunk
        {"name": "read fp4 t100", "op": "read", "cache": "fp4", "tokens": 100, "kv_heads": 4, "dim": 512, "page": 16,
         "kv_shared": False, "k_exp": 0, "v_exp": -4},
        # a long request's rows in front of its prompt's next chunk
        {"name": "read fp4 t30000", "op": "read", "cache": "fp4", "tokens": 30000, "kv_heads": 4, "dim": 512,
         "page": 16, "kv_shared": False, "k_exp": 0, "v_exp": -4},
        # the same from an e4m3 cache, an odd count
        {"name": "read fp8 t20011", "op": "read", "cache": "fp8", "tokens": 20011, "kv_heads": 8, "dim": 256,
         "page": 32, "kv_shared": False, "k_exp": 0, "v_exp": 0},
        # a small batch over short contexts: the smallest decode
        {"name": "decode b8 l1024", "op": "decode", "batch": 8, "len_lo": 1024, "len_hi": 1024, "tokens": 1, "layer": 0,
         "page": 16, "window": 0, "kv_shared": False, "k_exp": 0, "v_exp": -4},
        # long contexts, a global layer
        {"name": "decode b4 l32768", "op": "decode", "batch": 4, "len_lo": 32768, "len_hi": 32768, "tokens": 1,
         "layer": 0, "page": 16, "window": 0, "kv_shared": False, "k_exp": 0, "v_exp": -4},
        # lengths from a thousand tokens to 128 thousand in one batch, K=V storage: the largest
        {"name": "decode kv b8 mixed", "op": "decode", "batch": 8, "len_lo": 1024, "len_hi": 131072, "tokens": 1,
         "layer": 0, "page": 16, "window": 0, "kv_shared": True, "k_exp": 0, "v_exp": 0},
        # a sliding-window layer of the same kind of batch, windows that start inside a page
        {"name": "decode window b61", "op": "decode", "batch": 61, "len_lo": 700, "len_hi": 20000, "tokens": 1,
         "layer": 2, "page": 16, "window": 1024, "kv_shared": False, "k_exp": 1, "v_exp": -2},
        # two query tokens a request (draft verification), six query heads on a KV head, odd lengths
        {"name": "decode t2 b13", "op": "decode", "batch": 13, "len_lo": 999, "len_hi": 9001, "tokens": 2, "layer": 4,
         "page": 32, "window": 0, "kv_shared": False, "k_exp": 0, "v_exp": -3},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("store", "read", "decode", "decode"))
    exps = {"k_exp": rng.choice((-1, 0, 2)), "v_exp": rng.choice((-5, -3, 0))}
    if op != "decode":
        heads, dim = rng.choice(((4, 512), (2, 512), (8, 256), (1, 256), (3, 256)))
        c = {"op": op, "tokens": _log(rng, 1, 24000), "kv_heads": heads, "dim": dim,
             "page": rng.choice((16, 32, 48, 64)), "kv_shared": rng.random() < 0.3, **exps}
        if op == "store":
            return {**c, "fused": rng.random() < 0.5, "padding": rng.choice((0.0, 0.05, 0.5))}
        return {**c, "cache": rng.choice(("fp4", "fp4", "fp8", "bf16"))}
    batch, layer = _log(rng, 1, 160), rng.randrange(len(LAYERS))
    hi = _log(rng, 4, max(8, min(131072, 120000 // batch)))
    return {"op": op, "batch": batch, "len_lo": max(4, hi // rng.choice((1, 2, 16))), "len_hi": max(4, hi),
            "tokens": rng.choice((1, 1, 1, 2, 4)), "layer": layer, "page": rng.choice((16, 32, 64)),
            "window": rng.choice((512, 1000, 1024)) if LAYERS[layer][2] == 256 and rng.random() < 0.6 else 0,
            "kv_shared": rng.random() < 0.3, **exps}


# ---- inputs -------------------------------------------------------------------


def _gen(seed, device="cpu"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _spread(n, lo, hi):
    """n whole numbers in [lo, hi], spread over their logarithm: a case's lengths, whatever the seed."""
    u = (torch.arange(n, dtype=torch.float64) + 0.5) / max(n, 1)
    return (lo * (max(hi, lo) / lo) ** u).round().to(torch.int64).clamp(lo, max(lo, hi))


def _rows(shape, exp, g):
    """bf16 rows as a projection gives them: a few dims (the same in every row) many times the others."""
    x = torch.randn(shape, generator=g, device="cuda")
    big = torch.rand(shape[-1], generator=g, device="cuda") < 0.03
    return (x * torch.where(big, 6.0, 1.0) * 2.0 ** exp).to(torch.bfloat16)


def _slots_of_run(n, page, g, spare):
    """Slots of n tokens that lie one behind another in shuffled pages, and how many pages there are."""
    pages = (n + page - 1) // page + spare
    perm = torch.randperm(pages, generator=g)
    at = torch.arange(n) + int(torch.randint(0, page, (1,), generator=g))
    return perm[at // page] * page + at % page, pages


def _desc(c, heads, dim, pages, kind):
    from paged_gqa_decode_global_gb300 import binding as b
    return b.layer_desc(heads, heads, dim, c["page"], pages, pages, 0, c["kv_shared"],
                        {"fp4": b.PD_KV_FP4_E2M1, "fp8": b.PD_KV_FP8_E4M3, "bf16": b.PD_KV_BF16}[kind])


def _random_pool(pages, heads, page, dim, exp, g):
    """A 4-bit pool in use: (codes, block scales) of quantised rows."""
    return _plain_quantise(_rows((pages, heads, page, dim), exp, g), exp)


def _prepare_store(c, seed):
    g, dg = _gen(seed), _gen(seed, "cuda")
    n, H, d, P = c["tokens"], c["kv_heads"], c["dim"], c["page"]
    slots, pages = _slots_of_run(n, P, g, 3)
    slots[torch.rand(n, generator=g) < c["padding"]] = -1
    width = 3 if c["fused"] else 1  # a fused projection's row holds other heads too
    k = _rows((n, width * H, d), c["k_exp"], dg)[:, :H]
    v = None if c["kv_shared"] else _rows((n, width * H, d), c["v_exp"], dg)[:, (width - 1) * H:]
    s = {"k": k, "v": v, "slots": slots.to(torch.int32).cuda()}
    s["kp"], s["ks"] = _random_pool(pages, H, P, d, c["k_exp"], dg)
    s["vp"], s["vs"] = (None, None) if v is None else _random_pool(pages, H, P, d, c["v_exp"], dg)
    s["ko"] = torch.zeros((n, H, d), dtype=torch.bfloat16, device="cuda")
    s["vo"] = None if v is None else torch.zeros_like(s["ko"])
    s["flags"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        s["desc"] = _desc(c, H, d, pages, "fp4")
    return s


def _prepare_read(c, seed):
    g, dg = _gen(seed), _gen(seed, "cuda")
    n, H, d, P = c["tokens"], c["kv_heads"], c["dim"], c["page"]
    slots, pages = _slots_of_run(n, P, g, 3)
    s = {"slots": slots.to(torch.int32).cuda(), "cache": c["cache"], "ks": None, "vs": None, "vp": None}
    for name in ("k",) if c["kv_shared"] else ("k", "v"):
        if c["cache"] == "fp4":
            s[name + "p"], s[name + "s"] = _random_pool(pages, H, P, d, c[name + "_exp"], dg)
        else:
            x = _rows((pages, H, P, d), c[name + "_exp"], dg)
            if c["cache"] == "fp8":
                scale = x.float().abs().amax(dim=(2, 3)) / 448.0
                x = (x.float() / scale[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8)
                s[name + "s"] = scale
            s[name + "p"] = x
    s["ko"] = torch.zeros((n, H, d), dtype=torch.bfloat16, device="cuda")
    s["vo"] = None if c["kv_shared"] else torch.zeros_like(s["ko"])
    s["flags"] = torch.zeros(1, dtype=torch.int32, device="cuda")
    if own:
        s["desc"] = _desc(c, H, d, pages, c["cache"])
    return s


def _lens(c):
    """Cached tokens of each request, the new ones counted."""
    return _spread(c["batch"], max(c["len_lo"], c["tokens"]), max(c["len_hi"], c["tokens"]))


def _span(c):
    """Attended tokens of each request: all, or the union of its query tokens' windows."""
    lens = _lens(c)
    return lens if not c["window"] else torch.minimum(lens, torch.tensor(c["window"] + c["tokens"] - 1))


def _prepare_decode(c, seed):
    g, dg = _gen(seed), _gen(seed, "cuda")
    Hq, H, d = LAYERS[c["layer"]]
    B, T, P = c["batch"], c["tokens"], c["page"]
    lens = _lens(c)[torch.randperm(B, generator=g)]
    held = (lens + P - 1) // P
    pages, width = int(held.sum()) + 5, int(held.max())
    perm = torch.randperm(pages, generator=g)
    at, first = torch.arange(width), torch.cumsum(held, 0) - held
    table = torch.where(at[None] < held[:, None], perm[(first[:, None] + at[None]).clamp(max=pages - 1)], -1)
    q = (torch.randn((B, T, Hq, d), generator=dg, device="cuda") * 2.0 ** -c["k_exp"]).to(torch.bfloat16)
    s = {"q": q if T > 1 else q.view(B, Hq, d), "table": table.to(torch.int32).cuda(),
         "lens": lens.to(torch.int32).cuda(), "span": int(_span(c).max()), "window": c["window"], "tokens": T,
         "scale": 1.0 / math.sqrt(d)}
    s["kp"], s["ks"] = _random_pool(pages, H, P, d, c["k_exp"], dg)
    s["vp"], s["vs"] = (None, None) if c["kv_shared"] else _random_pool(pages, H, P, d, c["v_exp"], dg)
    s["out"] = torch.zeros_like(s["q"])
    if own:
        from paged_gqa_decode_global_gb300 import binding as b
        s["step"] = b.LayerStep(Hq, H, d, P, pages, width, lens.tolist(), window=c["window"],
                                kv_shared=c["kv_shared"], kv_dtype=b.PD_KV_FP4_E2M1, query_tokens=T)
    return s


def prepare(case, seed):
    s = {"store": _prepare_store, "read": _prepare_read, "decode": _prepare_decode}[case["op"]](case, seed)
    s.update(op=case["op"], k_exp=case["k_exp"], v_exp=case["k_exp"] if case["kv_shared"] else case["v_exp"])
    return s


# ---- the plain forms ------------------------------------------------------------


def _plain_quantise(rows, exp):
    """[..., d] rows -> codes [..., d / 2], e4m3 scales as bytes [..., d / 16]. In 32 bits: a bf16 is 8 bits and a scale 4
    wide, so a quotient that is not on a border is further from it than 32 bits round."""
    x = (rows.float() * 2.0 ** -exp).unflatten(-1, (-1, BLOCK))
    scale = (x.abs().amax(-1) / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn)
    s = scale.float().unsqueeze(-1)
    y = torch.where(s > 0, x / s, torch.zeros_like(x))
    a = y.abs()
    # to the nearest e2m1, a value halfway to the even code
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5.0))
    code = (code + (y < 0).to(torch.uint8) * 8).flatten(-2)
    return code[..., ::2] + code[..., 1::2] * 16, scale.view(torch.uint8)


def _values(codes, scales, exp):
    """The values that codes under block scales stand for, in fp32."""
    lut = torch.tensor(E2M1 + tuple(-v for v in E2M1), device=codes.device)
    i = torch.arange(256, device=codes.device)
    pairs = torch.stack([lut[i % 16], lut[i // 16]], -1)
    x = pairs[codes.int()].flatten(-2).unflatten(-1, (-1, BLOCK))
    return (x * (scales.view(torch.float8_e4m3fn).float() * 2.0 ** exp).unsqueeze(-1)).flatten(-2)


def _read_rows(s, name, slot, cache):
    pool, scale = s[name + "p"], s[name + "s"]
    P = pool.shape[2]
    page, off = slot // P, slot % P
    if cache == "fp4":
        return _values(pool[page, :, off], scale[page, :, off], s[name + "_exp"])
    x = pool[page, :, off]
    return x.view(torch.float8_e4m3fn).float() * scale[page][:, :, None] if cache == "fp8" else x


def _plain_store(s):
    slot = s["slots"].long()
    keep = torch.nonzero(slot >= 0).squeeze(1)
    slot, P = slot[keep], s["kp"].shape[2]
    page, off = slot // P, slot % P

    def put(name):
        codes, scales = _plain_quantise(s[name][keep], s[name + "_exp"])
        s[name + "p"][page, :, off] = codes
        s[name + "s"][page, :, off] = scales
        s[name + "o"][keep] = _read_rows(s, name, slot, "fp4").to(torch.bfloat16)

    put("k")
    if s["v"] is not None:
        put("v")
    return _rows_out(s)


def _plain_read(s):
    slot = s["slots"].long()
    s["ko"] = _read_rows(s, "k", slot, s["cache"]).to(torch.bfloat16)
    if s["vp"] is not None:
        s["vo"] = _read_rows(s, "v", slot, s["cache"]).to(torch.bfloat16)
    return _rows_out(s)


def _rows_out(s):
    return {"k": s["ko"]} if s["vo"] is None else {"k": s["ko"], "v": s["vo"]}


def _plain_decode(s):
    q, T, table = s["q"], s["tokens"], s["table"].long()
    B, Hq, d = q.shape[0], q.shape[-2], q.shape[-1]
    H, P = s["kp"].shape[1], s["kp"].shape[2]
    lens, dev = s["lens"].long(), q.device
    end = lens[:, None] - T + 1 + torch.arange(T, device=dev)  # of each query token's positions
    lo = (end - s["window"]).clamp(min=0) if s["window"] else torch.zeros_like(end)
    pos = lo[:, :1] + torch.arange(s["span"], device=dev)
    slot = torch.gather(table, 1, (pos // P).clamp(max=table.shape[1] - 1)).clamp(min=0) * P + pos % P
    k = _read_rows(s, "k", slot, "fp4").transpose(1, 2)
    v = k if s["vp"] is None else _read_rows(s, "v", slot, "fp4").transpose(1, 2)
    qf = q.float().view(B, T, H, Hq // H, d).permute(0, 2, 1, 3, 4)
    w = torch.matmul(qf.reshape(B, H, -1, d), k.transpose(2, 3)) * s["scale"]
    mask = (pos[:, None] >= end[:, :, None]) | (pos[:, None] < lo[:, :, None])
    w = w.view(B, H, T, Hq // H, -1).masked_fill_(mask[:, None, :, None], -math.inf)
    w = torch.exp(w - w.amax(-1, keepdim=True))
    o = torch.matmul(w.view(B, H, -1, w.shape[-1]), v).view(B, H, T, Hq // H, d) / w.sum(-1, keepdim=True)
    s["out"] = o.permute(0, 2, 1, 3, 4).reshape(q.shape).to(torch.bfloat16)
    return s["out"]


# ---- one pass -------------------------------------------------------------------


def run(state):
    s = state
    if not own:
        return {"store": _plain_store, "read": _plain_read, "decode": _plain_decode}[s["op"]](s)
    from paged_gqa_decode_global_gb300 import binding as b
    if s["op"] == "decode":
        return s["step"](s["q"], s["kp"], s["vp"], s["table"], s["lens"], s["scale"], s["out"], k_scale=s["ks"],
                         v_scale=s["vs"], k_exp=s["k_exp"], v_exp=s["v_exp"])
    if s["op"] == "store":
        b.paged_decode_write_slots_fp4(s["desc"], s["k"], s["v"], s["slots"], s["kp"], s["vp"], s["ks"], s["vs"],
                                       s["flags"], k_exp=s["k_exp"], v_exp=s["v_exp"])
    if s["op"] == "store" or s["cache"] == "fp4":
        b.paged_decode_read_slots_fp4(s["desc"], s["slots"], s["kp"], s["vp"], s["ks"], s["vs"], s["ko"], s["vo"],
                                      s["flags"], k_exp=s["k_exp"], v_exp=s["v_exp"])
    elif s["cache"] == "fp8":
        b.paged_decode_read_slots_fp8(s["desc"], s["slots"], s["kp"], s["vp"], s["ks"], s["vs"], s["ko"], s["vo"],
                                      s["flags"])
    else:
        b.paged_decode_read_slots(s["desc"], s["slots"], s["kp"], s["vp"], s["ko"], s["vo"], s["flags"])
    return _rows_out(s)


def work(case):
    c = case
    if c["op"] == "decode":
        Hq, H, d = LAYERS[c["layer"]]
        span, rows = float(_span(c).sum()), c["batch"] * c["tokens"] * Hq
        row = H * (d // 2 + d // BLOCK) * (1 if c["kv_shared"] else 2)
        # each query row's own positions
        own_span = float(_span(c).sum()) - c["batch"] * (c["tokens"] - 1) / 2
        return {"bytes": span * row + 4 * rows * d, "flops": 4 * c["tokens"] * Hq * d * own_span}
    parts, d = c["kv_heads"] * (1 if c["kv_shared"] else 2), c["dim"]
    packed = d // 2 + d // BLOCK
    if c["op"] == "store":
        rows = c["tokens"] * (1 - c["padding"]) * parts
        return {"bytes": rows * (2 * d + packed + 2 * d) + 4 * c["tokens"], "flops": 0}
    held = {"fp4": packed, "fp8": d, "bf16": 2 * d}[c["cache"]]
    return {"bytes": c["tokens"] * (parts * (held + 2 * d) + 4), "flops": 0}


# ---- the definitions in 64 bits ---------------------------------------------------


def _nearest(x, grid):
    """Each x's nearest value of a rising grid, the one of even index where two are equally near."""
    hi = torch.searchsorted(grid, x).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = x - grid[lo], grid[hi] - x
    even = torch.where(lo % 2 == 0, lo, hi)
    return grid[torch.where(below < above, lo, torch.where(above < below, hi, even))]


def _exact_round_trip(rows, exp):
    """What a row stands for once it has been held in 4 bits."""
    x = rows.double() / 2.0 ** exp
    e, m = torch.meshgrid(torch.arange(16), torch.arange(8), indexing="ij")
    e4m3 = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10).double()).flatten()[:-1].double().to(x.device)
    e2m1 = torch.tensor(E2M1, dtype=torch.float64, device=x.device)
    b = x.view(*x.shape[:-1], -1, BLOCK)
    s = _nearest(b.abs().max(-1, keepdim=True).values / 6.0, e4m3)
    held = torch.sign(b) * _nearest(b.abs() / torch.where(s > 0, s, torch.ones_like(s)), e2m1) * s
    return held.view(x.shape) * 2.0 ** exp


def _exact_values(s, name, cache, page, off):
    """Rows at (page, off) of a pool, by the definition of its type."""
    pool, scale = s[name + "p"][page, :, off], s[name + "s"]
    if cache == "bf16":
        return pool.double()
    if cache == "fp8":
        return pool.view(torch.float8_e4m3fn).double() * scale[page].double()[..., None]
    code = torch.stack([pool & 15, pool >> 4], -1).flatten(-2).long()
    mag, sign = code & 7, 1.0 - 2.0 * (code >> 3)
    half = torch.where(mag < 2, mag, (2 + mag % 2) << (mag // 2 - 1).clamp(min=0)).double()  # in units of a half
    each = scale[page, :, off].view(torch.float8_e4m3fn).double().repeat_interleave(BLOCK, -1)
    return sign * half / 2 * each * 2.0 ** s[name + "_exp"]


def _exact_store(s):
    got, on = {}, s["slots"] >= 0
    for name in ("k",) if s["v"] is None else ("k", "v"):
        got[name] = s[name + "o"].double()
        got[name][on] = _exact_round_trip(s[name][on], s[name + "_exp"])
    return got


def _exact_read(s):
    slot, P = s["slots"].long(), s["kp"].shape[2]
    names = ("k",) if s["vp"] is None else ("k", "v")
    return {n: _exact_values(s, n, s["cache"], slot // P, slot % P) for n in names}


def _exact_decode(s):
    q, T, P = s["q"], s["tokens"], s["kp"].shape[2]
    B, Hq, d, H = q.shape[0], q.shape[-2], q.shape[-1], s["kp"].shape[1]
    out = torch.zeros((B, T, Hq, d), dtype=torch.float64, device=q.device)
    for b, L in enumerate(s["lens"].tolist()):
        first = max(0, L - T + 1 - s["window"]) if s["window"] else 0
        pos = torch.arange(first, L, device=q.device)
        page = s["table"][b].long()[pos // P]
        k = _exact_values(s, "k", "fp4", page, pos % P)
        v = k if s["vp"] is None else _exact_values(s, "v", "fp4", page, pos % P)
        qb = q.view(B, T, H, Hq // H, d)[b].double()
        w = torch.einsum("thgd,nhd->thgn", qb, k) * s["scale"]
        last = L - T + torch.arange(T, device=q.device)[:, None]
        seen = (pos <= last) & ((pos > last - s["window"]) if s["window"] else True)
        w.masked_fill_(~seen[:, None, None], -math.inf)
        out[b] = torch.einsum("thgn,nhd->thgd", torch.softmax(w, -1), v).reshape(T, Hq, d)
    return out.view(q.shape)


def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "read": _exact_read, "decode": _exact_decode}[case["op"]](s)
