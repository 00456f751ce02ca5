"""The serving operators around decode attention over a paged cache, as cases that can be timed and compared.

Three operators that one step of a serving loop runs behind one another:
  slots   block tables and slot maps of a batch's new tokens, built on the GPU from the requests' lengths
  write   the new tokens' K / V rows into their slots of the paged cache (bf16, or e4m3 under the pages' scales)
  shared  decode attention of a batch whose requests share long prefixes, each prefix's rows read once for all of them

With `own` false, run() computes an operator in its plain form from elementary torch operations; with `own` true it
makes the calls a user makes of the framework.
"""
import math

import torch

own = False

# query heads, KV heads, head_dim of the layer kinds served here
LAYERS = ((16, 4, 512), (8, 2, 512), (16, 8, 256), (32, 4, 256), (24, 4, 512))


def listed():
    return [
        # one decode step of a busy server: every request gets one token, few need a page
        {"name": "slots decode b256", "op": "slots", "batch": 256, "page": 16, "new_lo": 1, "new_hi": 1,
         "cached_hi": 4096, "idle": 0.0},
        # decode steps and prompt chunks in one batch, an odd number of requests
        {"name": "slots mixed b1001", "op": "slots", "batch": 1001, "page": 32, "new_lo": 1, "new_hi": 600,
         "cached_hi": 3000, "idle": 0.3},
        # a wave of long prompts
        {"name": "slots prompts b48", "op": "slots", "batch": 48, "page": 64, "new_lo": 700, "new_hi": 32000,
         "cached_hi": 0, "idle": 0.0},
        # one decode step's rows, where latency counts
        {"name": "write decode t64", "op": "write", "tokens": 64, "kv_heads": 4, "dim": 512, "page": 16,
         "fp8": False, "kv_shared": False, "fused": True, "padding": 0.0},
        # a prompt's rows out of a fused QKV projection
        {"name": "write prompt t16384", "op": "write", "tokens": 16384, "kv_heads": 4, "dim": 512, "page": 16,
         "fp8": False, "kv_shared": False, "fused": True, "padding": 0.0},
        # ragged chunks padded to a fixed count, into an e4m3 cache
        {"name": "write fp8 t20011", "op": "write", "tokens": 20011, "kv_heads": 8, "dim": 256, "page": 32,
         "fp8": True, "kv_shared": False, "fused": False, "padding": 0.1},
        # two samples of one short prompt: the smallest call
        {"name": "shared b2 p1024", "op": "shared", "batch": 2, "groups": 1, "prefix": 1024, "own_hi": 60,
         "tokens": 1, "layer": 0, "page": 16, "fp8": False, "kv_shared": False},
        # sixteen requests under one long document
        {"name": "shared b16 p32768", "op": "shared", "batch": 16, "groups": 1, "prefix": 32768, "own_hi": 500,
         "tokens": 1, "layer": 0, "page": 16, "fp8": False, "kv_shared": False},
        # K=V storage, a system prompt under many requests
        {"name": "shared kv b64 p8192", "op": "shared", "batch": 64, "groups": 1, "prefix": 8192, "own_hi": 400,
         "tokens": 1, "layer": 0, "page": 16, "fp8": False, "kv_shared": True},
        # an e4m3 cache
        {"name": "shared fp8 b32 p32768", "op": "shared", "batch": 32, "groups": 1, "prefix": 32768, "own_hi": 700,
         "tokens": 1, "layer": 0, "page": 16, "fp8": True, "kv_shared": False},
        # several prompts in one batch, two query tokens a request (draft verification), odd lengths
        {"name": "shared groups b45 t2", "op": "shared", "batch": 45, "groups": 5, "prefix": 4000, "own_hi": 333,
         "tokens": 2, "layer": 2, "page": 32, "fp8": False, "kv_shared": False},
        # the largest: a full batch under one long prompt
        {"name": "shared b256 p16384", "op": "shared", "batch": 256, "groups": 1, "prefix": 16384, "own_hi": 256,
         "tokens": 1, "layer": 0, "page": 16, "fp8": False, "kv_shared": False},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(("slots", "write", "shared", "shared"))
    if op == "slots":
        batch = _log(rng, 1, 1500)
        hi = max(1, min(32000, 1400000 // batch))
        new_hi = _log(rng, 1, hi)
        return {"op": op, "batch": batch, "page": rng.choice((16, 32, 48, 64, 128)),
                "new_lo": rng.randint(1, new_hi), "new_hi": new_hi,
                "cached_hi": rng.choice((0, _log(rng, 1, 6000))), "idle": rng.choice((0.0, 0.2))}
    if op == "write":
        heads, dim = rng.choice(((4, 512), (2, 512), (8, 256), (1, 256), (8, 128), (3, 128)))
        return {"op": op, "tokens": _log(rng, 1, 20000), "kv_heads": heads, "dim": dim,
                "page": rng.choice((16, 32, 48, 64)), "fp8": dim > 128 and rng.random() < 0.4,
                "kv_shared": rng.random() < 0.3, "fused": rng.random() < 0.5, "padding": rng.choice((0.0, 0.05, 0.5))}
    batch = _log(rng, 1, 200)
    groups, tokens = min(batch, rng.choice((1, 1, 2, 3, 7))), rng.choice((1, 1, 1, 2, 3))
    # the rows and the prefixes together stay within the largest listed case
    prefix = _log(rng, 16, max(64, min(40000, 16384 * 128 // (batch * groups * tokens))))
    return {"op": op, "batch": batch, "groups": groups, "prefix": prefix, "own_hi": _log(rng, 1, 500),
            "tokens": tokens, "layer": rng.randrange(len(LAYERS)), "page": rng.choice((16, 32, 64)),
            "fp8": rng.random() < 0.35, "kv_shared": rng.random() < 0.35}


# ---- inputs -------------------------------------------------------------------


def _gen(seed, device="cpu"):
    g = torch.Generator(device=device)
    g.manual_seed(seed)
    return g


def _spread(n, lo, hi):
    """n whole numbers in [lo, hi], spread over their logarithm: a case's lengths, whatever the seed."""
    u = (torch.arange(n, dtype=torch.float64) + 0.5) / max(n, 1)
    return (lo * (max(hi, lo) / lo) ** u).round().to(torch.int64).clamp(lo, max(lo, hi))


def _new_tokens(c):
    new = _spread(c["batch"], c["new_lo"], c["new_hi"])
    idle = int(c["idle"] * c["batch"])
    if idle:
        new[torch.linspace(0, c["batch"] - 1, idle).long()] = 0
    return new


def _prefix_pages(c):
    """The first group's prefix the longest, the others' spread below it; whole pages."""
    whole = max(1, c["prefix"] // c["page"])
    return torch.cat([torch.tensor([whole]), _spread(c["groups"] - 1, max(1, whole // 8), whole)])


def _own_lens(c):
    return _spread(c["batch"], c["tokens"], max(c["tokens"], c["own_hi"]))


def _shuffled(x, g):
    return x[torch.randperm(x.numel(), generator=g)]


def _quantise(x):
    """[pages, heads, P, d] -> e4m3 codes as bytes, and the scale of each (page, head)."""
    scale = x.float().abs().amax(dim=(2, 3)) / 448.0
    return (x.float() / scale[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), scale


def _tables(pages_of, perm):
    """Pages handed out in order from `perm`: [n, widest] int32, -1 past a row's last."""
    n, width = len(pages_of), max(1, int(pages_of.max()))
    first = torch.cumsum(pages_of, 0) - pages_of
    at = torch.arange(width)
    idx = (first[:, None] + at[None]).clamp(max=perm.numel() - 1)
    return torch.where(at[None] < pages_of[:, None], perm[idx], torch.full((1,), -1)).to(torch.int32)


def _prepare_slots(c, seed):
    g = _gen(seed)
    B, P = c["batch"], c["page"]
    new = _shuffled(_new_tokens(c), g)
    cached = torch.randint(0, c["cached_hi"] + 1, (B,), generator=g)
    held = (cached + P - 1) // P
    need = (cached + new + P - 1) // P - held
    total = int(held.sum() + need.sum())
    pool = total + 16
    perm = torch.randperm(pool, generator=g)
    width = (c["cached_hi"] + c["new_hi"] + P - 1) // P + 2
    table = torch.full((B, width), -1, dtype=torch.int32)
    t = _tables(held, perm)
    table[:, :t.shape[1]] = torch.where(t[:, :width] >= 0, t[:, :width], table[:, :t.shape[1]])
    tokens = int(new.sum())
    dev = "cuda"
    free = perm[int(held.sum()):].to(torch.int32)
    taken = 5 if free.numel() >= int(need.sum()) + 5 else 0  # earlier calls took some
    s = {"cached": cached.to(torch.int32).to(dev), "new": new.to(torch.int32).to(dev), "table": table.to(dev),
         "free": free.to(dev), "range": torch.tensor([taken, free.numel()], dtype=torch.int32, device=dev),
         "page": P, "pool": pool, "max_tokens": tokens + 3,
         "lens": torch.zeros(B, dtype=torch.int32, device=dev),
         "starts": torch.zeros(B + 1, dtype=torch.int32, device=dev),
         "slots": torch.zeros(tokens + 3, dtype=torch.int32, device=dev),
         "positions": torch.zeros(tokens + 3, dtype=torch.int32, device=dev),
         "range_out": torch.zeros(2, dtype=torch.int32, device=dev),
         "flags": torch.zeros(1, dtype=torch.int32, device=dev)}
    if own:
        from paged_gqa_decode_global_gb300 import binding as b
        s["workspace"] = torch.zeros(b.paged_decode_append_slots_workspace(B), dtype=torch.uint8, device=dev)
    return s


def _prepare_write(c, seed):
    g, dg = _gen(seed), _gen(seed, "cuda")
    n, H, d, P = c["tokens"], c["kv_heads"], c["dim"], c["page"]
    pages = (n + P - 1) // P + 3
    dev = "cuda"
    # rows land in runs of consecutive slots of shuffled pages, as a prompt's do
    perm = torch.randperm(pages, generator=g)
    at = torch.arange(n) + int(torch.randint(0, P, (1,), generator=g))
    slots = perm[at // P] * P + at % P
    slots[torch.rand(n, generator=g) < c["padding"]] = -1
    width = (3 if c["fused"] else 1) * H * d  # a fused projection's row holds other heads too
    k = torch.randn((n, width), generator=dg, device=dev).to(torch.bfloat16)[:, :H * d].view(n, H, d)
    v = None if c["kv_shared"] else \
        torch.randn((n, width), generator=dg, device=dev).to(torch.bfloat16)[:, width - H * d:].view(n, H, d)
    kp = torch.randn((pages, H, P, d), generator=dg, device=dev).to(torch.bfloat16)
    vp = None if c["kv_shared"] else torch.randn((pages, H, P, d), generator=dg, device=dev).to(torch.bfloat16)
    s = {"k": k, "v": v, "kp": kp, "vp": vp, "ks": None, "vs": None, "slots": slots.to(torch.int32).to(dev),
         "flags": torch.zeros(1, dtype=torch.int32, device=dev), "fp8": c["fp8"]}
    if c["fp8"]:
        s["kp"], s["ks"] = _quantise(kp)
        if vp is not None:
            s["vp"], s["vs"] = _quantise(vp)
    if own:
        from paged_gqa_decode_global_gb300 import binding as b
        s["desc"] = b.layer_desc(H, H, d, P, pages, pages, 0, c["kv_shared"],
                                 b.PD_KV_FP8_E4M3 if c["fp8"] else b.PD_KV_BF16)
    return s


def _prepare_shared(c, seed):
    g, dg = _gen(seed), _gen(seed, "cuda")
    Hq, Hkv, d = LAYERS[c["layer"]]
    B, T, P, n = c["batch"], c["tokens"], c["page"], c["groups"]
    dev = "cuda"
    pages = _prefix_pages(c)
    cuts = torch.randperm(B - 1, generator=g)[:n - 1].sort().values + 1 if n > 1 else torch.zeros(0, dtype=torch.int64)
    starts = torch.cat([torch.zeros(1, dtype=torch.int64), cuts, torch.tensor([B])])
    own_lens = _shuffled(_own_lens(c), g)
    own_pages = (own_lens + P - 1) // P
    total = int(pages.sum() + own_pages.sum())
    perm = torch.randperm(total + 7, generator=g)
    ptab = _tables(pages, perm)
    table = _tables(own_pages, perm[int(pages.sum()):])
    q = (torch.randn((B, T, Hq, d), generator=dg, device=dev) * 1.5).to(torch.bfloat16)
    if T == 1:
        q = q.view(B, Hq, d)
    kp = torch.randn((total + 7, Hkv, P, d), generator=dg, device=dev).to(torch.bfloat16)
    vp = None if c["kv_shared"] else torch.randn((total + 7, Hkv, P, d), generator=dg, device=dev).to(torch.bfloat16)
    s = {"q": q, "kp": kp, "vp": vp, "ks": None, "vs": None, "ptab": ptab.to(dev), "table": table.to(dev),
         "plens": (pages * P).to(torch.int32).to(dev), "lens": own_lens.to(torch.int32).to(dev),
         "starts": starts.to(torch.int32).to(dev), "scale": 1.0 / math.sqrt(d), "tokens": T,
         "rows": int((starts[1:] - starts[:-1]).max()), "out": torch.zeros_like(q)}
    if c["fp8"]:
        s["kp"], s["ks"] = _quantise(kp)
        if vp is not None:
            s["vp"], s["vs"] = _quantise(vp)
    if own:
        from paged_gqa_decode_global_gb300 import binding as b
        s["step"] = b.SharedPrefixStep(Hq, Hkv, d, P, total + 7, table.shape[1], own_lens.tolist(),
                                       group_starts=starts.tolist(), prefix_lens=(pages * P).tolist(),
                                       max_prefix_pages=ptab.shape[1], kv_shared=c["kv_shared"],
                                       kv_dtype=b.PD_KV_FP8_E4M3 if c["fp8"] else b.PD_KV_BF16, query_tokens=T)
    return s


def prepare(case, seed):
    s = {"slots": _prepare_slots, "write": _prepare_write, "shared": _prepare_shared}[case["op"]](case, seed)
    s["op"] = case["op"]
    return s


# ---- the plain forms ------------------------------------------------------------


def _plain_slots(s):
    P, cap = s["page"], s["max_tokens"]
    cached, new, table = s["cached"].long(), s["new"].long(), s["table"]
    B, width = table.shape
    held = (cached + P - 1) // P
    need = (cached + new + P - 1) // P - held
    starts = torch.cat([new.new_zeros(1), torch.cumsum(new, 0)])
    first = s["range"][0].long() + torch.cumsum(need, 0) - need
    # new pages into the tables
    req = torch.repeat_interleave(torch.arange(B, device=new.device), need)
    k = torch.arange(req.numel(), device=new.device) - (torch.cumsum(need, 0) - need)[req]
    table[req, held[req] + k] = s["free"][first[req] + k]
    # the tokens' positions and slots
    req = torch.repeat_interleave(torch.arange(B, device=new.device), new)
    pos = cached[req] + torch.arange(req.numel(), device=new.device) - starts[req]
    slot = table[req, pos // P].long() * P + pos % P
    pad = new.new_full((cap - req.numel(),), -1)
    s["slots"] = torch.cat([slot, pad]).to(torch.int32)
    s["positions"] = torch.cat([pos, pad]).to(torch.int32)
    s["starts"] = starts.to(torch.int32)
    s["lens"] = (cached + new).to(torch.int32)
    s["range_out"] = torch.stack([s["range"][0] + need.sum().to(torch.int32), s["range"][1]])
    return _slots_out(s)


def _slots_out(s):
    return {"table": s["table"], "lens": s["lens"], "starts": s["starts"], "slots": s["slots"],
            "positions": s["positions"], "range": s["range_out"]}


def _plain_write(s):
    P = s["kp"].shape[2]
    slot = s["slots"].long()
    keep = torch.nonzero(slot >= 0).squeeze(1)
    page, off = slot[keep] // P, slot[keep] % P

    def put(pool, rows, scale):
        x = rows[keep]
        if s["fp8"]:
            x = (x.float() / scale[page][:, :, None]).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        pool[page, :, off] = x

    put(s["kp"], s["k"], s["ks"])
    if s["vp"] is not None:
        put(s["vp"], s["v"], s["vs"])
    return _write_out(s)


def _write_out(s):
    # an e4m3 cache's values, as the type that holds them
    f = (lambda p: p.view(torch.float8_e4m3fn)) if s["fp8"] else (lambda p: p)
    return {"k": f(s["kp"])} if s["vp"] is None else {"k": f(s["kp"]), "v": f(s["vp"])}


def _rows_of(pool, scale, table):
    """[n, tokens, Hkv, d] in fp32: the rows behind a table (entries past a row's last page are page 0's, masked later)."""
    idx = table.long().clamp(min=0)
    x = pool[idx]
    x = x.view(torch.float8_e4m3fn).float() * scale[idx][:, :, :, None, None] if scale is not None else x.float()
    n, m, H, P, d = x.shape
    return x.permute(0, 1, 3, 2, 4).reshape(n, m * P, H, d)


def _plain_shared(s):
    q, T = s["q"], s["tokens"]
    B, Hq, d = q.shape[0], q.shape[-2], q.shape[-1]
    Hkv = s["kp"].shape[1]
    G, R = Hq // Hkv, s["rows"]
    dev = q.device
    starts = s["starts"].long()
    N = starts.numel() - 1
    qf = q.float().view(B, T, Hkv, G, d)
    # requests of a group side by side, padded to the largest group
    at = starts[:-1, None] + torch.arange(R, device=dev)
    here = at < starts[1:, None]
    qg = qf[at.clamp(max=B - 1)].permute(0, 3, 1, 2, 4, 5).reshape(N, Hkv, R * T * G, d)
    k = _rows_of(s["kp"], s["ks"], s["ptab"]).permute(0, 2, 1, 3)
    v = k if s["vp"] is None else _rows_of(s["vp"], s["vs"], s["ptab"]).permute(0, 2, 1, 3)
    sp = torch.matmul(qg, k.transpose(2, 3)) * s["scale"]
    sp.masked_fill_((torch.arange(k.shape[2], device=dev) >= s["plens"].long()[:, None])[:, None, None], -math.inf)
    mp = sp.amax(-1, keepdim=True)
    ep = torch.exp(sp - mp)
    del sp
    lp, op = ep.sum(-1, keepdim=True), torch.matmul(ep, v)
    del ep, k, v

    def back(x):
        """[N, Hkv, R*T*G, e] -> [B, T, Hkv, G, e]"""
        return x.view(N, Hkv, R, T, G, -1).permute(0, 2, 3, 1, 4, 5)[here]

    mp, lp, op = back(mp), back(lp), back(op)
    # each request's own tokens, causal among the new ones
    k = _rows_of(s["kp"], s["ks"], s["table"]).permute(0, 2, 1, 3)
    v = k if s["vp"] is None else _rows_of(s["vp"], s["vs"], s["table"]).permute(0, 2, 1, 3)
    so = torch.matmul(qf.permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, d), k.transpose(2, 3)) * s["scale"]
    so = so.view(B, Hkv, T, G, -1).permute(0, 2, 1, 3, 4)
    end = s["lens"].long()[:, None] - T + 1 + torch.arange(T, device=dev)
    mask = torch.arange(so.shape[-1], device=dev) >= end[:, :, None]
    so = so.masked_fill(mask[:, :, None, None], -math.inf)
    m = torch.maximum(mp, so.amax(-1, keepdim=True))
    eo, wp = torch.exp(so - m), torch.exp(mp - m)
    oo = torch.matmul(eo.permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, -1), v)
    oo = oo.view(B, Hkv, T, G, d).permute(0, 2, 1, 3, 4)
    o = (wp * op + oo) / (wp * lp + eo.sum(-1, keepdim=True))
    s["out"] = o.reshape(q.shape).to(torch.bfloat16)
    return s["out"]


# ---- one pass -------------------------------------------------------------------


def run(state):
    s = state
    if not own:
        return {"slots": _plain_slots, "write": _plain_write, "shared": _plain_shared}[s["op"]](s)
    from paged_gqa_decode_global_gb300 import binding as b
    if s["op"] == "slots":
        b.paged_decode_append_slots(s["page"], s["pool"], s["cached"], s["new"], s["free"], s["range"], s["table"],
                                    s["lens"], s["starts"], s["slots"], s["positions"], s["range_out"], s["flags"],
                                    s["workspace"])
        return _slots_out(s)
    if s["op"] == "write":
        if s["fp8"]:
            b.paged_decode_write_slots_fp8(s["desc"], s["k"], s["v"], s["slots"], s["kp"], s["vp"], s["ks"], s["vs"],
                                           s["flags"])
        else:
            b.paged_decode_write_slots(s["desc"], s["k"], s["v"], s["slots"], s["kp"], s["vp"], s["flags"])
        return _write_out(s)
    return s["step"](s["q"], s["kp"], s["vp"], s["ptab"], s["plens"], s["starts"], s["table"], s["lens"], s["scale"],
                     s["out"], k_scale=s["ks"], v_scale=s["vs"])


def work(case):
    c = case
    if c["op"] == "slots":
        new = _new_tokens(c)
        tokens, pages = int(new.sum()), int(new.sum()) / c["page"]
        return {"bytes": 8 * tokens + 8 * pages + 16 * c["batch"], "flops": 0}
    if c["op"] == "write":
        rows = c["tokens"] * (1 - c["padding"]) * c["kv_heads"] * (1 if c["kv_shared"] else 2)
        return {"bytes": rows * c["dim"] * (2 + (1 if c["fp8"] else 2)) + 4 * c["tokens"], "flops": 0}
    Hq, Hkv, d = LAYERS[c["layer"]]
    prefix, lens = float(_prefix_pages(c).sum()) * c["page"], float(_own_lens(c).sum())
    row = Hkv * d * (1 if c["fp8"] else 2) * (1 if c["kv_shared"] else 2)
    rows = c["batch"] * c["tokens"] * Hq
    return {"bytes": (prefix + lens) * row + 4 * rows * d,
            "flops": 4 * rows * d * (prefix / c["groups"] + lens / c["batch"])}


# ---- the definitions in 64 bits ---------------------------------------------------


def _exact_slots(s):
    cached, new, free = (s[k].tolist() for k in ("cached", "new", "free"))
    table, P, at = s["table"].tolist(), s["page"], int(s["range"][0])
    starts, slots, positions = [0], [], []
    for b, (have, n) in enumerate(zip(cached, new)):
        for pos in range(have, have + n):
            if pos % P == 0:
                table[b][pos // P] = free[at]
                at += 1
            slots.append(table[b][pos // P] * P + pos % P)
            positions.append(pos)
        starts.append(len(slots))
    pad = [-1] * (s["max_tokens"] - len(slots))
    i = lambda v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    return {"table": i(table), "lens": i([a + n for a, n in zip(cached, new)]), "starts": i(starts),
            "slots": i(slots + pad), "positions": i(positions + pad), "range": i([at, int(s["range"][1])])}


def _exact_write(s):
    P = s["kp"].shape[2]
    got = {}
    for name in ("k", "v"):
        pool, rows, scale = s[name + "p"], s[name], s[name + "s"]
        if pool is None:
            continue
        x = (pool.view(torch.float8_e4m3fn) if s["fp8"] else pool).double()
        flat = x.permute(0, 2, 1, 3).reshape(-1, x.shape[1], x.shape[3])  # by slot
        slot = s["slots"].long()
        on = slot >= 0
        y = rows.double()
        if s["fp8"]:
            per = scale.double().repeat_interleave(P, 0)  # [slots, heads]
            y = (y / per[slot.clamp(min=0)][:, :, None]).clamp(-448, 448)
        flat[slot[on]] = y[on]
        got[name] = flat.view(x.shape[0], P, x.shape[1], x.shape[3]).permute(0, 2, 1, 3)
    return got


def _exact_shared(s):
    q, T, scale = s["q"], s["tokens"], s["scale"]
    B, Hq, d = q.shape[0], q.shape[-2], q.shape[-1]
    pools = [(s["kp"], s["ks"])] + ([(s["vp"], s["vs"])] if s["vp"] is not None else [])
    Hkv, P = s["kp"].shape[1], s["kp"].shape[2]
    starts = s["starts"].tolist()
    out = torch.zeros((B, T, Hq, d), dtype=torch.float64, device=q.device)

    def rows(pool, ps, table, n):
        pages = table[: (n + P - 1) // P].long()
        x = (pool[pages].view(torch.float8_e4m3fn) if ps is not None else pool[pages]).double()
        if ps is not None:
            x = x * ps[pages].double()[:, :, None, None]
        return x.transpose(1, 2).reshape(-1, Hkv, d)[:n]

    for n in range(len(starts) - 1):
        head = [rows(p, ps, s["ptab"][n], int(s["plens"][n])) for p, ps in pools]
        for b in range(starts[n], starts[n + 1]):
            L = int(s["lens"][b])
            tail = [rows(p, ps, s["table"][b], L) for p, ps in pools]
            full = [torch.cat([x, y]) for x, y in zip(head, tail)]
            k, v = full[0], full[-1]
            qb = q.view(B, T, Hkv, Hq // Hkv, d)[b].double()
            w = torch.einsum("thgd,nhd->thgn", qb, k) * scale
            last = len(k) - T + torch.arange(T, device=q.device)
            w.masked_fill_((torch.arange(len(k), device=q.device) > last[:, None])[:, None, None], -math.inf)
            out[b] = torch.einsum("thgn,nhd->thgd", torch.softmax(w, -1), v).reshape(T, Hq, d)
    return out.view(q.shape)


def exact(case, seed):
    s = prepare(case, seed)
    return {"slots": _exact_slots, "write": _exact_write, "shared": _exact_shared}[case["op"]](s)
