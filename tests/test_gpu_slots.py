"""Block tables and slot maps built on the GPU against a plain Python statement
of the rules (whole numbers: equal), and the write of rows into those slots
(bf16: the same bits; e4m3: the quotient in fp32, rounded by torch)."""
import random

import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b

pytestmark = pytest.mark.gpu


def _expect(P, num_pages, cap_pages, max_tokens, cached, new, free, rng, table):
    """The header's rules, one request after another."""
    table = [list(r) for r in table]
    lo, end = max(0, rng[0]), min(len(free), rng[1])
    end = max(end, lo)
    at, taken, tok, flags = lo, lo, 0, 0
    lens, starts, slots, pos = [], [], [-1] * max_tokens, [-1] * max_tokens
    for r, (c, n) in enumerate(zip(cached, new)):
        ok = c >= 0 and n >= 0 and c + n <= cap_pages * P
        width = n if 0 <= n <= cap_pages * P else 0
        need = -(-(c + n) // P) - -(-c // P) if ok else 0
        starts.append(tok)
        tok += width
        at += need
        if not ok or tok > max_tokens:
            flags |= b.PD_DEVFLAG_BAD_SEQLEN
            ok = False
        elif need and at > end:
            flags |= b.PD_DEVFLAG_NO_PAGES
            ok = False
        lens.append(c + n if ok else c)
        if not ok:
            continue
        taken = at if need else taken
        for k in range(need):
            table[r][-(-c // P) + k] = free[at - need + k]
        for j in range(n):
            page = table[r][(c + j) // P]
            pos[starts[r] + j] = c + j
            if 0 <= page < num_pages:
                slots[starts[r] + j] = page * P + (c + j) % P
            else:
                flags |= b.PD_DEVFLAG_BAD_PAGE
    return dict(table=table, lens=lens, starts=starts + [tok], slots=slots, pos=pos, rng=[taken, end], flags=flags)


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def _run(P, num_pages, max_tokens, cached, new, free, rng, table, in_place=False, positions=True, ws=None):
    B, width = len(cached), len(table[0]) if table else 1
    t = _i32(table).view(B, width)
    c, fr = _i32(cached), _i32(rng)
    lens = c if in_place else torch.full((B,), -7, dtype=torch.int32, device="cuda")
    fro = fr if in_place else torch.full((2,), -7, dtype=torch.int32, device="cuda")
    starts = torch.full((B + 1,), -7, dtype=torch.int32, device="cuda")
    # one entry past the end shows a write out of range
    slots = torch.full((max_tokens + 1,), -77, dtype=torch.int32, device="cuda")
    pos = torch.full((max_tokens + 1,), -77, dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    if ws is None:
        ws = torch.zeros(b.paged_decode_append_slots_workspace(B), dtype=torch.uint8, device="cuda")
    b.paged_decode_append_slots(P, num_pages, c, _i32(new), _i32(free), fr, t, lens, starts, slots[:max_tokens],
                                pos[:max_tokens] if positions else None, fro, flags, ws)
    torch.cuda.synchronize()
    assert int(slots[-1]) == -77 and int(pos[-1]) == -77
    return dict(table=t.tolist(), lens=lens.tolist(), starts=starts.tolist(), slots=slots[:-1].tolist(),
                pos=pos[:-1].tolist(), rng=fro.tolist(), flags=int(flags))


def _case(rng, B, P, cached_hi, new_hi, extra=3, short=0, idle=0.2):
    cached = [rng.randint(0, cached_hi) for _ in range(B)]
    new = [0 if rng.random() < idle else rng.randint(1, new_hi) for _ in range(B)]
    held = [-(-c // P) for c in cached]
    need = sum(-(-(c + n) // P) - h for c, n, h in zip(cached, new, held))
    width = max([1] + [-(-(c + n) // P) for c, n in zip(cached, new)]) + 1
    pages = list(range(sum(held) + need + extra))
    rng.shuffle(pages)
    table, at = [], 0
    for h in held:
        table.append(pages[at:at + h] + [-1] * (width - h))
        at += h
    free = pages[at:]
    return dict(P=P, num_pages=len(pages) or 1, max_tokens=sum(new) + extra, cached=cached, new=new, free=free,
                rng=[0, len(free) - short], table=table)


def _check(c, **kw):
    e = _expect(c["P"], c["num_pages"], len(c["table"][0]) if c["table"] else 1, c["max_tokens"], c["cached"],
                c["new"], c["free"], c["rng"], c["table"])
    g = _run(**c, **kw)
    if kw.get("positions") is False:
        e.pop("pos"), g.pop("pos")
    for k in e:
        assert g[k] == e[k], k
    return e


@pytest.mark.parametrize("B,P,cached_hi,new_hi", [
    (1, 16, 0, 1), (1, 16, 40, 700), (7, 16, 100, 1), (256, 16, 500, 1), (33, 48, 90, 5), (1023, 32, 60, 9),
    (1024, 16, 0, 20), (1025, 16, 31, 3), (3000, 64, 200, 2), (9, 1, 7, 9), (40, 128, 1000, 2500), (5, 16, 0, 9001)])
@pytest.mark.parametrize("in_place", [False, True])
def test_append_slots(B, P, cached_hi, new_hi, in_place):
    rng = random.Random(B * 7 + P)
    e = _check(_case(rng, B, P, cached_hi, new_hi), in_place=in_place)
    assert e["flags"] == 0


@pytest.mark.parametrize("seed", range(6))
def test_append_slots_with_too_few_pages(seed):
    rng = random.Random(seed)
    c = _case(rng, rng.choice((3, 60, 1500)), 16, 50, 40, extra=0, short=0)
    c["rng"] = [0, len(c["free"]) * 2 // 3]
    e = _check(c, in_place=bool(seed & 1), positions=seed != 3)
    short = len(c["free"]) > c["rng"][1]  # the list held exactly what they need
    assert bool(e["flags"] & b.PD_DEVFLAG_NO_PAGES) == short


def test_append_slots_bad_lengths():
    rng = random.Random(5)
    c = _case(rng, 50, 16, 60, 30)
    cap = len(c["table"][0]) * 16
    c["new"][3], c["new"][11], c["new"][12], c["new"][20] = -4, cap + 1, 2 ** 31 - 1, cap
    c["cached"][30] = -1
    c["cached"][31] = 2 ** 31 - 1
    e = _check(c)
    assert e["flags"] & b.PD_DEVFLAG_BAD_SEQLEN


@pytest.mark.parametrize("cut", [0, 1, 57])
def test_append_slots_tokens_past_the_slot_map(cut):
    c = _case(random.Random(cut), 60, 16, 60, 30)
    c["max_tokens"] = sum(c["new"]) * cut // 60
    e = _check(c)
    assert e["flags"] & b.PD_DEVFLAG_BAD_SEQLEN


def test_append_slots_bad_pages():
    c = _case(random.Random(9), 20, 16, 60, 30, idle=0.0)
    c["free"][2], c["free"][3] = -1, c["num_pages"]
    r = next(i for i, x in enumerate(c["cached"]) if x % 16)
    c["table"][r][c["cached"][r] // 16] = c["num_pages"] + 5
    e = _check(c)
    assert e["flags"] & b.PD_DEVFLAG_BAD_PAGE and not e["flags"] & b.PD_DEVFLAG_NO_PAGES


@pytest.mark.parametrize("rng", [[-5, 3], [2, 10 ** 6], [7, 2], [400, 500]])
def test_append_slots_free_range_is_cut_to_the_list(rng):
    c = _case(random.Random(4), 12, 16, 20, 12, idle=0.0)
    c["rng"] = rng
    _check(c)


def test_append_slots_empty_batch_and_no_tokens():
    _check(dict(P=16, num_pages=4, max_tokens=3, cached=[], new=[], free=[1], rng=[0, 1], table=[]))
    _check(dict(P=16, num_pages=4, max_tokens=0, cached=[5], new=[0], free=[1], rng=[0, 1], table=[[2]]))


def test_append_slots_grows_a_cache_step_by_step_in_a_graph():
    """In place, captured once and replayed: 40 decode steps equal the rules step by step."""
    P, B, width = 16, 5, 8
    cached, table, free = [0, 3, 15, 16, 17], [[-1] * width for _ in range(B)], list(range(60))
    random.Random(1).shuffle(free)
    at = 0
    for r, c in enumerate(cached):
        for k in range(-(-c // P)):
            table[r][k] = free[at]
            at += 1
    state = dict(c=_i32(cached), t=_i32(table), fr=_i32([at, 60]), new=_i32([1, 1, 2, 1, 1]))
    starts, slots = torch.zeros(B + 1, dtype=torch.int32, device="cuda"), torch.zeros(8, dtype=torch.int32, device="cuda")
    flags, fl = torch.zeros(1, dtype=torch.int32, device="cuda"), _i32(free)
    ws = torch.zeros(b.paged_decode_append_slots_workspace(B), dtype=torch.uint8, device="cuda")

    def call():
        b.paged_decode_append_slots(P, 60, state["c"], state["new"], fl, state["fr"], state["t"], state["c"], starts,
                                    slots, None, state["fr"], flags, ws)

    keep = [x.clone() for x in (state["c"], state["t"], state["fr"])]
    s = torch.cuda.Stream()
    with torch.cuda.stream(s):
        call()  # warm-up
        s.synchronize()
        for x, k in zip((state["c"], state["t"], state["fr"]), keep):
            x.copy_(k)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            call()
    torch.cuda.synchronize()
    rng = [at, 60]
    for _ in range(40):
        g.replay()
        torch.cuda.synchronize()
        e = _expect(P, 60, width, 8, cached, [1, 1, 2, 1, 1], free, rng, table)
        cached, table, rng = e["lens"], e["table"], e["rng"]
        assert state["c"].tolist() == cached and state["t"].tolist() == table and state["fr"].tolist() == rng
        assert slots.tolist() == e["slots"] and int(flags) == e["flags"] == 0


# ---- the cache write --------------------------------------------------------------


def _bits(t):
    return t.view(torch.int16) if t.dtype == torch.bfloat16 else t


def _write_case(n, H, d, P, fp8, kvs, pad, seed, fused):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    pages = -(-n // P) + 2
    slots = torch.randperm(pages * P, device="cuda", generator=g)[:n].to(torch.int32)
    slots[torch.rand(n, device="cuda", generator=g) < pad] = -1
    w = (H + 1) * d if fused else H * d
    mk = lambda: torch.randn(n, w, device="cuda", generator=g).to(torch.bfloat16)[:, w - H * d:].view(n, H, d)  # noqa: E731
    k, v = mk(), None if kvs else mk()
    if fp8:
        pool = lambda: torch.randint(0, 120, (pages, H, P, d), device="cuda", generator=g).to(torch.uint8)  # noqa: E731
    else:
        pool = lambda: torch.randn(pages, H, P, d, device="cuda", generator=g).to(torch.bfloat16)  # noqa: E731
    kp, vp = pool(), None if kvs else pool()
    sc = lambda: torch.rand(pages, H, device="cuda", generator=g) * 0.02 + 1e-3  # noqa: E731
    ks, vs = (sc(), None if kvs else sc()) if fp8 else (None, None)
    return slots, k, v, kp, vp, ks, vs


def _plain_write(pool, rows, slots, scale, P):
    out = pool.clone()
    on = (slots >= 0) & (slots < pool.shape[0] * P)
    s = slots[on].long()
    x = rows[on]
    if scale is not None:
        x = (x.float() / scale[s // P][:, :, None]).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
    out[s // P, :, s % P] = x
    return out


@pytest.mark.parametrize("n,H,d,P,fp8,kvs,fused", [
    (1, 4, 512, 16, False, False, False), (1, 1, 128, 16, False, True, True), (5, 8, 256, 48, False, False, True),
    (333, 3, 128, 16, False, False, True), (2000, 4, 512, 64, False, True, False), (1, 2, 256, 16, True, False, False),
    (77, 8, 256, 32, True, False, True), (1025, 4, 512, 16, True, True, False), (130, 5, 512, 1, False, False, False)])
@pytest.mark.parametrize("pad", [0.0, 0.3])
def test_write_slots(n, H, d, P, fp8, kvs, fused, pad):
    slots, k, v, kp, vp, ks, vs = _write_case(n, H, d, P, fp8, kvs, pad, n + d, fused)
    ek = _plain_write(kp, k, slots, ks, P)
    ev = None if kvs else _plain_write(vp, v, slots, vs, P)
    desc = b.layer_desc(H, H, d, P, kp.shape[0], 8, 0, kvs, b.PD_KV_FP8_E4M3 if fp8 else b.PD_KV_BF16)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    if fp8:
        b.paged_decode_write_slots_fp8(desc, k, v, slots, kp, vp, ks, vs, flags)
    else:
        b.paged_decode_write_slots(desc, k, v, slots, kp, vp, flags)
    torch.cuda.synchronize()
    assert int(flags) == 0
    assert torch.equal(_bits(kp), _bits(ek))
    assert kvs or torch.equal(_bits(vp), _bits(ev))


def test_write_slots_bad_slots_are_skipped_and_flagged():
    slots, k, v, kp, vp, _, _ = _write_case(40, 4, 512, 16, False, False, 0.0, 3, False)
    slots[[1, 7, 30]] = torch.tensor([-2, kp.shape[0] * 16, 2 ** 31 - 1], dtype=torch.int32, device="cuda")
    ek, ev = _plain_write(kp, k, slots, None, 16), _plain_write(vp, v, slots, None, 16)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.paged_decode_write_slots(b.layer_desc(4, 4, 512, 16, kp.shape[0], 8), k, v, slots, kp, vp, flags)
    torch.cuda.synchronize()
    assert int(flags) == b.PD_DEVFLAG_BAD_PAGE
    assert torch.equal(_bits(kp), _bits(ek)) and torch.equal(_bits(vp), _bits(ev))


def test_write_slots_fp8_special_values():
    """Infinities clamp, NaN stays NaN, a zero scale saturates (0 / 0 is NaN), ties go to even."""
    vals = [float("inf"), float("-inf"), float("nan"), 0.0, -0.0, 448.0, 1e30, -1e30, 17.0, 19.0, 2 ** -10, 3 * 2 ** -10,
            2 ** -9, 464.0, 465.0, 0.4375]
    k = torch.tensor(vals, device="cuda").to(torch.bfloat16).repeat(8 * 2).view(2, 1, 128)
    kp = torch.zeros(2, 1, 16, 128, dtype=torch.uint8, device="cuda")
    ks = torch.tensor([[1.0], [0.0]], device="cuda")
    slots = torch.tensor([3, 16], dtype=torch.int32, device="cuda")
    ek = _plain_write(kp, k, slots, ks, 16)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.paged_decode_write_slots_fp8(b.layer_desc(1, 1, 128, 16, 2, 8, 0, True, b.PD_KV_FP8_E4M3), k, None, slots, kp,
                                   None, ks, None, flags)
    got, exp = (x.view(torch.float8_e4m3fn).float() for x in (kp, ek))
    assert torch.equal(got.isnan(), exp.isnan())
    assert torch.equal(got.nan_to_num(7.0), exp.nan_to_num(7.0))


def test_write_slots_past_32_bit_offsets():
    """A pool of over 2^32 bytes: the last page's rows land at their place."""
    P, H, d = 16, 4, 512
    pages = (1 << 32) // (P * H * d * 2) + 9
    kp = torch.zeros(pages, H, P, d, dtype=torch.bfloat16, device="cuda")
    k = torch.randn(3, H, d, device="cuda").to(torch.bfloat16)
    slots = torch.tensor([pages * P - 1, 5, (pages - 7) * P], dtype=torch.int32, device="cuda")
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.paged_decode_write_slots(b.layer_desc(H, H, d, P, pages, 8, 0, True), k, None, slots, kp, None, flags)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(kp[s // P, :, s % P], k[i])
    assert int(kp.view(torch.int16).ne(0).any(-1).sum()) == 3 * H
