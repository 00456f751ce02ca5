"""Rows quantised into a 4-bit cache as they are written, against exact arithmetic (equal codes and scales), and cached
rows read back (equal values)."""
import math

import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b

pytestmark = pytest.mark.gpu

E2M1 = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)
E4M3 = torch.arange(0x7F, dtype=torch.uint8).view(torch.float8_e4m3fn).double()  # 0 .. 448


def nearest(x, grid):
    """Index of each x's (>= 0) nearest value of a rising grid, the even one where two are equally near."""
    hi = torch.searchsorted(grid, x.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    below, above = x - grid[lo], grid[hi] - x
    return torch.where(below < above, lo, torch.where(above < below, hi, torch.where(lo % 2 == 0, lo, hi)))


def quantise(rows, exp):
    """The header's rule in 64 bits: (codes [..., d / 2], scales [..., d / 16]) as bytes."""
    x = (rows.double().cpu() * 2.0 ** -exp).unflatten(-1, (-1, 16))
    amax = x.abs().amax(-1)
    s = nearest(amax.nan_to_num(nan=0.0, posinf=1e300) / 6, E4M3)
    nan = amax.isnan()
    v = E4M3[s].unsqueeze(-1)
    mag = x.abs().nan_to_num(nan=0.0, posinf=1e300) / torch.where(v > 0, v, torch.ones_like(v))
    code = nearest(mag, E2M1.contiguous()) + 8 * (torch.signbit(x)).long()
    code = torch.where((v > 0) & ~nan.unsqueeze(-1), code, torch.zeros_like(code)).flatten(-2)
    return ((code[..., ::2] + 16 * code[..., 1::2]).to(torch.uint8).cuda(),
            torch.where(nan, 0x7F, s).to(torch.uint8).cuda())


def values(codes, scales, exp):
    lut = torch.cat([E2M1, -E2M1]).to(codes.device)
    x = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    return x * (scales.view(torch.float8_e4m3fn).double() * 2.0 ** exp).repeat_interleave(16, -1)


def by_slot(pool):
    """[pages, H, P, e] -> [slots, H, e]"""
    return pool.transpose(1, 2).reshape(-1, pool.shape[1], pool.shape[3])


class Pools:
    def __init__(self, pages, H, P, d, kvs=False, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        r = lambda e: torch.randint(0, 256, (pages, H, P, e), generator=g, device="cuda", dtype=torch.uint8)  # noqa: E731
        self.kc, self.ks = r(d // 2), r(d // 16)
        self.vc, self.vs = (None, None) if kvs else (r(d // 2), r(d // 16))
        self.desc = b.layer_desc(H, H, d, P, pages, pages, 0, kvs, b.PD_KV_FP4_E2M1)
        self.flags = torch.zeros(1, dtype=torch.int32, device="cuda")

    def write(self, k, v, slots, **kw):
        b.paged_decode_write_slots_fp4(self.desc, k, v, slots, self.kc, self.vc, self.ks, self.vs, self.flags, **kw)

    def read(self, slots, k, v, **kw):
        b.paged_decode_read_slots_fp4(self.desc, slots, self.kc, self.vc, self.ks, self.vs, k, v, self.flags, **kw)


def special_rows(n, H, d, exp, seed):
    """Rows with blocks that go wrong easily: values halfway between codes, zeros, tiny ones, huge ones, NaN, infinity."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn((n, H, d), generator=g) * torch.exp(torch.randn((n, H, 1), generator=g) * 3)
    blk = x.view(-1, 16)
    for i in range(0, blk.shape[0], 3):
        s = float(E4M3[1 + (i * 7) % 126])
        mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0])
        blk[i] = torch.cat([mids, -mids]) * s
    blk[1::29] = 0.0
    blk[4::31] = -0.0
    blk[5::31] *= 2.0 ** -20
    blk[2::37] *= 2.0 ** 60
    blk[7::41] = 2.0 ** -9 * 3  # around the smallest scale's border
    blk[8::41] = 2.0 ** -9 * 6
    x = (x * 2.0 ** exp).to(torch.bfloat16)
    blk = x.view(-1, 16)
    blk[10::53, 3] = math.nan
    blk[11::53, 9] = math.inf
    blk[12::53, 15] = -math.inf
    return x.cuda()


@pytest.mark.parametrize("n", [1, 2, 31, 300, 5000])
@pytest.mark.parametrize("H,d,P", [(4, 512, 16), (2, 256, 48), (5, 256, 32), (1, 256, 16), (9, 512, 64)])
@pytest.mark.parametrize("kvs", [False, True])
def test_write_and_read_back(n, H, d, P, kvs):
    exps = {"k_exp": -3, "v_exp": -3 if kvs else 5}
    pages = -(-n // P) + 2
    pools = Pools(pages, H, P, d, kvs, seed=n)
    g = torch.Generator().manual_seed(n)
    slots = torch.randperm(pages * P, generator=g)[:n].to(torch.int32)
    slots[torch.rand(n, generator=g) < 0.1] = -1
    k = special_rows(n, H, d, exps["k_exp"], n)
    v = None if kvs else special_rows(n, H, d, exps["v_exp"], n + 1)
    before = [p.clone() for p in (pools.kc, pools.ks, pools.vc, pools.vs) if p is not None]
    dev = slots.cuda()
    pools.write(k, v, dev, **exps)
    on = slots >= 0
    at = slots[on].long().cuda()
    want = [by_slot(x).clone() for x in before]
    for i, (rows, e) in enumerate([(k, exps["k_exp"])] + ([] if kvs else [(v, exps["v_exp"])])):
        codes, scales = quantise(rows[on.cuda()], e)
        got_codes, got_scales = by_slot((pools.kc, pools.vc)[i]), by_slot((pools.ks, pools.vs)[i])
        want[2 * i][at], want[2 * i + 1][at] = codes, scales
        assert torch.equal(got_scales, want[2 * i + 1])
        # a NaN block's codes may be anything
        same = (got_codes == want[2 * i]).view(*got_codes.shape[:-1], -1, 8).all(-1)
        assert bool((same | (want[2 * i + 1] == 0x7F)).all())
    # and the way back, into strided rows; the skipped ones stay
    out = torch.full((n, 3 * H, d), 9.0, dtype=torch.bfloat16, device="cuda")
    ko, vo = out[:, H:2 * H], None if kvs else out[:, 2 * H:]
    pools.read(dev, ko, vo, **exps)
    assert int(pools.flags) == 0 and bool((out[:, :H] == 9.0).all())
    for rows, i, e in [(ko, 0, exps["k_exp"])] + ([] if kvs else [(vo, 1, exps["v_exp"])]):
        exact = values(by_slot((pools.kc, pools.vc)[i])[at], by_slot((pools.ks, pools.vs)[i])[at], e)
        got = rows[on.cuda()]
        nan = exact.isnan()
        assert torch.equal(got.isnan(), nan) and torch.equal(got.double()[~nan], exact[~nan])
        assert bool((rows[~on.cuda()] == 9.0).all())


@pytest.mark.parametrize("exp", [-64, -10, 0, 11, 64])
def test_every_bf16_under_every_scale(exp):
    """All bf16 values below a scale's reach, each with the scale that its block's largest sets."""
    vals = torch.arange(0x7F80, dtype=torch.int32).to(torch.int16).view(torch.bfloat16).double() * 2.0 ** -exp
    rows = []
    for s in E4M3[1:].tolist():
        x = vals[(vals >= s * 2.0 ** -3) & (vals < s * 6.0)]
        x = x[torch.randperm(len(x), generator=torch.Generator().manual_seed(1))[:900]]
        x = torch.cat([x, x.new_zeros(-len(x) % 15)]).view(-1, 15)
        rows.append(torch.cat([x.new_full((x.shape[0], 1), 6.0 * s), x], 1))
    x = (torch.cat(rows) * 2.0 ** exp).to(torch.bfloat16)
    x = torch.cat([x, x.new_zeros((-x.shape[0] % 16, 16))]).view(-1, 1, 256).cuda()
    n = x.shape[0]
    pools = Pools(-(-n // 16), 1, 16, 256, True)
    pools.write(x, None, torch.arange(n, dtype=torch.int32, device="cuda"), k_exp=exp, v_exp=exp)
    codes, scales = quantise(x, exp)
    assert torch.equal(by_slot(pools.ks)[:n], scales)
    assert torch.equal(by_slot(pools.kc)[:n], codes)


@pytest.mark.parametrize("n", [1, 37, 4000])
@pytest.mark.parametrize("H,d,P", [(4, 512, 16), (8, 256, 32), (3, 128, 48)])
@pytest.mark.parametrize("kvs", [False, True])
@pytest.mark.parametrize("fp8", [False, True])
def test_read_bf16_and_e4m3(n, H, d, P, kvs, fp8):
    g = torch.Generator(device="cuda").manual_seed(n)
    pages = -(-n // P) + 1
    make = lambda: torch.randn((pages, H, P, d), generator=g, device="cuda").to(torch.bfloat16)  # noqa: E731
    pools, scales = [make() for _ in range(1 if kvs else 2)], [None, None]
    exact = [by_slot(p).double() for p in pools]
    if fp8:
        scales = [torch.rand((pages, H), generator=g, device="cuda") * 3 + 1e-3 for _ in pools] + [None]
        pools = [p.to(torch.float8_e4m3fn).view(torch.uint8) for p in pools]
        exact = [by_slot((p.view(torch.float8_e4m3fn).float() * s[:, :, None, None])).double()
                 for p, s in zip(pools, scales)]
    slots = torch.randint(0, pages * P, (n,), generator=g, device="cuda", dtype=torch.int32)  # (repeats are fine)
    slots[n // 2] = -1 if n > 1 else slots[0]
    out = [torch.full((n, H, d), 5.0, dtype=torch.bfloat16, device="cuda") for _ in pools] + [None]
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    desc = b.layer_desc(H, H, d, P, pages, pages, 0, kvs, b.PD_KV_FP8_E4M3 if fp8 else b.PD_KV_BF16)
    pools.append(None)
    if fp8:
        b.paged_decode_read_slots_fp8(desc, slots, pools[0], pools[1], scales[0], scales[1], out[0], out[1], flags)
    else:
        b.paged_decode_read_slots(desc, slots, pools[0], pools[1], out[0], out[1], flags)
    assert int(flags) == 0
    for o, e in zip(out, exact):
        want = torch.where((slots >= 0)[:, None, None], e[slots.long().clamp(min=0)].to(torch.bfloat16),
                           torch.full_like(o, 5.0))
        assert torch.equal(o, want)


def test_bad_slots_are_reported_and_touch_nothing():
    pools = Pools(4, 2, 16, 256, seed=1)
    k = torch.randn((5, 2, 256), device="cuda").to(torch.bfloat16)
    before = [x.clone() for x in (pools.kc, pools.ks, pools.vc, pools.vs)]
    for bad in (64, -2, 2 ** 31 - 1, -2 ** 31):
        slots = torch.tensor([-1, bad, -1, bad, -1], dtype=torch.int32, device="cuda")
        pools.write(k, k, slots)
        assert int(pools.flags) == b.PD_DEVFLAG_BAD_PAGE
        assert all(torch.equal(x, y) for x, y in zip(before, (pools.kc, pools.ks, pools.vc, pools.vs)))
        pools.flags.zero_()
        out = torch.full((5, 2, 256), 3.0, dtype=torch.bfloat16, device="cuda")
        pools.read(slots, out, torch.empty_like(out))
        assert int(pools.flags) == b.PD_DEVFLAG_BAD_PAGE and bool((out == 3.0).all())
        pools.flags.zero_()


def test_offsets_past_32_bits():
    """A pool whose bytes pass 2^32: rows at its end."""
    H, P, d = 8, 64, 512
    pages = (2 ** 32 // (H * P * d // 2)) + 3
    pools = Pools(1, H, P, d, True)
    pools.desc.num_pages = pages
    pools.kc = torch.zeros((pages, H, P, d // 2), dtype=torch.uint8, device="cuda")
    pools.ks = torch.zeros((pages, H, P, d // 16), dtype=torch.uint8, device="cuda")
    slots = torch.tensor([pages * P - 1, pages * P - 64 * 3, 5], dtype=torch.int32, device="cuda")
    k = special_rows(3, H, d, 0, 2)
    pools.write(k, None, slots)
    codes, scales = quantise(k, 0)
    for i, s in enumerate(slots.tolist()):
        assert torch.equal(pools.ks[s // P, :, s % P], scales[i])
    out = torch.empty_like(k)
    pools.read(slots, out, None)
    want = values(codes, scales, 0)
    nan = want.isnan()
    assert torch.equal(out.double()[~nan], want[~nan]) and torch.equal(out.isnan(), nan)


def test_written_and_read_in_a_captured_graph():
    pools = Pools(20, 4, 16, 512, seed=3)
    k = torch.randn((100, 4, 512), device="cuda").to(torch.bfloat16)
    slots = torch.randperm(320, device="cuda")[:100].to(torch.int32)
    out = [torch.empty_like(k), torch.empty_like(k)]
    pools.write(k, k, slots)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pools.write(k, k, slots)
        pools.read(slots, *out)
    for seed in (1, 2, 3):
        k.copy_(torch.randn(k.shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda"))
        slots.copy_(torch.randperm(320, device="cuda")[:100])
        graph.replay()
        want = values(*quantise(k, 0), 0)
        assert torch.equal(out[0].double(), want) and torch.equal(out[1].double(), want)


def test_serving_steps():
    """Slots, quantised rows, decode over them and the read-back of a chunk, run behind one another with no host in
    between; the decode sees what is read back."""
    B, P, H, Hq, d, steps, cap = 5, 16, 4, 16, 512, 4, 400
    g = torch.Generator(device="cuda").manual_seed(5)
    width, pages = -(-cap // P), B * -(-cap // P)
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    pools = Pools(pages, H, P, d, seed=5)
    table = torch.full((B, width), -1, dtype=torch.int32, device="cuda")
    free = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
    rng, lens, starts = torch.tensor([0, pages], dtype=torch.int32, device="cuda"), i32(B), i32(B + 1)
    ws = torch.zeros(b.paged_decode_append_slots_workspace(B), dtype=torch.uint8, device="cuda")
    step = b.LayerStep(Hq, H, d, P, pages, width, [cap] * B, kv_dtype=b.PD_KV_FP4_E2M1)
    scale, k_exp, v_exp = 1 / math.sqrt(d), b.fp4_exponent(8.0), b.fp4_exponent(0.5)
    seen = [([], []) for _ in range(B)]
    outs = []
    for n in range(steps):
        new = [137, 1, 300, 16, 0] if n == 0 else [1] * B
        total = sum(new)
        slots, pos = i32(total), i32(total)
        b.paged_decode_append_slots(P, pages, lens, torch.tensor(new, dtype=torch.int32, device="cuda"), free, rng, table,
                                    lens, starts, slots, pos, rng, pools.flags, ws)
        k = torch.randn((total, H, d), generator=g, device="cuda").to(torch.bfloat16)
        v = (torch.randn((total, H, d), generator=g, device="cuda") * 0.05).to(torch.bfloat16)
        pools.write(k, v, slots, k_exp=k_exp, v_exp=v_exp)
        kb, vb = torch.empty_like(k), torch.empty_like(v)
        pools.read(slots, kb, vb, k_exp=k_exp, v_exp=v_exp)
        q = torch.randn((B, Hq, d), generator=g, device="cuda").to(torch.bfloat16)
        out = torch.empty_like(q)
        step(q, pools.kc, pools.vc, table, lens, scale, out, k_scale=pools.ks, v_scale=pools.vs, k_exp=k_exp, v_exp=v_exp)
        for r, (x, y) in enumerate(zip(kb.split(new), vb.split(new))):
            seen[r][0].append(x)
            seen[r][1].append(y)
        outs.append((q, out, [torch.cat(s[0]) for s in seen], [torch.cat(s[1]) for s in seen]))
    step.check()
    assert int(pools.flags) == 0
    for q, out, ks, vs in outs:
        for r in range(B):
            if not len(ks[r]):
                assert not out[r].any()
                continue
            w = torch.softmax(torch.einsum("hgd,nhd->hgn", q[r].double().view(H, -1, d), ks[r].double()) * scale, -1)
            want = torch.einsum("hgn,nhd->hgd", w, vs[r].double()).reshape(Hq, d)
            # the output's rounding to bf16, and f16's of the weights
            assert float((out[r].double() - want).norm() / want.norm()) < 2.0 ** -8 + 2.0 ** -10
