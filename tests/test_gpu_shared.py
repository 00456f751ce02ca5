"""Shared-prefix decode against attention over [prefix | own] in 64 bits.

Tolerance, element by element, from the roundings the kernels make (e = 2^-8,
half a bf16 step): the output's, e |out|; each probability's, rounded to bf16
(or, the FP8 own part, p times the V scale to f16: less, but for its subnormal
step 2^-25 of each code): e A, with A = softmax . |V|; a score's fp32 sum of d
products and its exponential's argument, both relative in p and so 2 ds A with
ds = scale * sum |q||k| * d 2^-24 + 4 (max |s| + 8) 2^-24; fp32 sums and merges of n terms,
at most n 2^-24 A each, taken as 2^-12 A for the lengths here.
"""
import math
import random

import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b

pytestmark = pytest.mark.gpu

E = torch.finfo(torch.bfloat16).eps / 2


def _quantise(x):
    s = x.float().abs().amax(dim=(2, 3)) / 448.0
    s = torch.where(s > 0, s, torch.ones_like(s))
    return (x.float() / s[:, :, None, None]).to(torch.float8_e4m3fn).view(torch.uint8), s


class Case:
    def __init__(self, Hq, Hkv, d, lens, starts, prefix, T=1, P=16, kvs=False, fp8=False, seed=0, q_std=1.0,
                 spare=3, garbage=True):
        g = torch.Generator().manual_seed(seed)
        dg = torch.Generator(device="cuda").manual_seed(seed)
        self.Hq, self.Hkv, self.d, self.T, self.P, self.kvs, self.fp8 = Hq, Hkv, d, T, P, kvs, fp8
        self.lens, self.starts, self.prefix = list(lens), list(starts), list(prefix)
        B, N = len(lens), len(prefix)
        pp, op = [n // P for n in prefix], [-(-n // P) for n in lens]
        total = sum(pp) + sum(op) + spare
        perm = torch.randperm(total, generator=g).tolist()
        w, ow = max(pp + [1]), max(op + [1])
        self.ptab, self.table, at = [], [], 0
        for n in pp:
            self.ptab.append(perm[at:at + n] + [-1] * (w - n))
            at += n
        for n in op:
            self.table.append(perm[at:at + n] + [-1] * (ow - n))
            at += n
        self.pages = total
        mk = lambda: torch.randn(total, Hkv, P, d, generator=dg, device="cuda").to(torch.bfloat16)  # noqa: E731
        self.kp, self.vp = mk(), None if kvs else mk()
        self.ks = self.vs = None
        if fp8:
            self.kp, self.ks = _quantise(self.kp)
            if not kvs:
                self.vp, self.vs = _quantise(self.vp)
        if garbage:  # what no request attends holds NaN: unused pages, and rows past the own tokens
            nan = 0x7f if fp8 else float("nan")
            for pool in (self.kp, self.vp):
                if pool is None:
                    continue
                if perm[at:]:
                    pool[torch.tensor(perm[at:], device="cuda")] = nan
                for r, n in enumerate(lens):
                    if n % P:
                        pool[self.table[r][n // P], :, n % P:] = nan
        self.q = (torch.randn((B, T, Hq, d) if T > 1 else (B, Hq, d), generator=dg, device="cuda") * q_std).to(
            torch.bfloat16)
        self.scale = 1.0 / math.sqrt(d)
        self.dev = dict(ptab=torch.tensor(self.ptab, dtype=torch.int32, device="cuda").view(N, w),
                        plens=torch.tensor(prefix, dtype=torch.int32, device="cuda"),
                        starts=torch.tensor(starts, dtype=torch.int32, device="cuda"),
                        table=torch.tensor(self.table, dtype=torch.int32, device="cuda").view(B, ow),
                        lens=torch.tensor(lens, dtype=torch.int32, device="cuda"))

    def step(self, **kw):
        a = dict(group_starts=self.starts, prefix_lens=self.prefix, max_prefix_pages=self.dev["ptab"].shape[1],
                 kv_shared=self.kvs, kv_dtype=b.PD_KV_FP8_E4M3 if self.fp8 else b.PD_KV_BF16, query_tokens=self.T)
        a.update(kw)
        return b.SharedPrefixStep(self.Hq, self.Hkv, self.d, self.P, self.pages, self.dev["table"].shape[1],
                                  a.pop("lens", self.lens), **a)

    def run(self, step=None, out=None):
        step = step or self.step()
        out = torch.full_like(self.q, float("nan")) if out is None else out
        v = self.dev
        step(self.q, self.kp, self.vp, v["ptab"], v["plens"], v["starts"], v["table"], v["lens"], self.scale, out,
             k_scale=self.ks, v_scale=self.vs)
        return out, step

    def _rows(self, pool, scale, pages, n):
        idx = torch.tensor(pages[:-(-n // self.P)], dtype=torch.long, device="cuda")
        x = pool[idx].view(torch.float8_e4m3fn).double() * scale[idx].double()[:, :, None, None] if self.fp8 \
            else pool[idx].double()
        return x.transpose(1, 2).reshape(-1, self.Hkv, self.d)[:n]

    def expect(self):
        """(out, tolerance) in 64 bits."""
        B, T, G = len(self.lens), self.T, self.Hq // self.Hkv
        o = torch.zeros(B, T, self.Hq, self.d, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(o)
        q = self.q.view(B, T, self.Hkv, G, self.d).double()
        for n in range(len(self.prefix)):
            for r in range(self.starts[n], self.starts[n + 1]):
                L = self.lens[r]
                kv = [torch.cat([self._rows(p, s, self.ptab[n], self.prefix[n]),
                                 self._rows(p, s, self.table[r], L)])
                      for p, s in ((self.kp, self.ks), (self.vp, self.vs)) if p is not None]
                k, v = kv[0], kv[-1]
                if not len(k):
                    continue
                s = torch.einsum("thgd,nhd->thgn", q[r], k) * self.scale
                a = torch.einsum("thgd,nhd->thgn", q[r].abs(), k.abs()) * abs(self.scale)
                last = len(k) - T + torch.arange(T, device="cuda")
                off = (torch.arange(len(k), device="cuda") > last[:, None])[:, None, None]
                w = torch.softmax(s.masked_fill(off, -math.inf), -1).nan_to_num(0.0)
                e = torch.einsum("thgn,nhd->thgd", w, v)
                A = torch.einsum("thgn,nhd->thgd", w, v.abs())
                ds = (a.masked_fill(off, 0).amax(-1) * self.d + 4 * (s.masked_fill(off, 0).abs().amax(-1) + 8)) * 2.0 ** -24
                t = E * e.abs() + (E + 2 * ds[..., None] + 2.0 ** -12) * A
                if self.fp8 and L:
                    codes = (self.kp if self.kvs else self.vp)[
                        torch.tensor(self.table[r][:-(-L // self.P)], device="cuda")]
                    c = codes.view(torch.float8_e4m3fn).double().nan_to_num(0.0).abs().sum((0, 2))  # [Hkv, d]
                    t = t + 2.0 ** -25 * c[:, None, :]
                o[r], tol[r] = e.reshape(T, self.Hq, self.d), t.reshape(T, self.Hq, self.d)
        return o.view(self.q.shape), tol.view(self.q.shape) + 1e-12

    def check(self, step=None):
        out, step = self.run(step)
        assert step.check() == 0
        e, tol = self.expect()
        assert torch.isfinite(out).all()
        over = ((out.double() - e).abs() / tol).max().item() if out.numel() else 0.0
        assert over <= 1.0, f"{over:.3f} of the tolerance"
        return out


LAYERS = [(16, 4, 512), (8, 2, 512), (4, 4, 512), (8, 1, 512), (12, 4, 512), (9, 1, 512), (32, 2, 512), (16, 8, 256),
          (32, 4, 256), (16, 1, 256), (8, 2, 128), (4, 4, 128)]


@pytest.mark.parametrize("Hq,Hkv,d", LAYERS)
@pytest.mark.parametrize("kvs", [False, True])
def test_layers(Hq, Hkv, d, kvs):
    Case(Hq, Hkv, d, [5, 1, 33, 16, 100], [0, 5], [400], kvs=kvs, seed=d + Hq).check()


@pytest.mark.parametrize("Hq,Hkv,d", [x for x in LAYERS if x[2] > 128])
@pytest.mark.parametrize("kvs", [False, True])
def test_layers_fp8(Hq, Hkv, d, kvs):
    Case(Hq, Hkv, d, [5, 1, 33, 16, 100], [0, 5], [400], kvs=kvs, fp8=True, seed=d + Hq).check()


@pytest.mark.parametrize("prefix", [16, 32, 112, 128, 144, 256, 272, 2000, 5008])
@pytest.mark.parametrize("fp8", [False, True])
def test_prefix_lengths(prefix, fp8):
    Case(16, 4, 512, [7, 40], [0, 2], [prefix], fp8=fp8, seed=prefix).check()


@pytest.mark.parametrize("batch", [1, 3, 4, 5, 8, 9, 16, 17, 33, 70])
@pytest.mark.parametrize("Hq,Hkv,d", [(16, 4, 512), (16, 8, 256)])
def test_batches(batch, Hq, Hkv, d):
    """Row tiles of 16 to 128 rows, full and cut."""
    rng = random.Random(batch)
    Case(Hq, Hkv, d, [rng.randint(1, 60) for _ in range(batch)], [0, batch], [640], seed=batch).check()


@pytest.mark.parametrize("P", [16, 32, 48, 64, 128, 256])
@pytest.mark.parametrize("fp8", [False, True])
def test_page_sizes(P, fp8):
    Case(16, 4, 512, [1, P + 3, 2 * P], [0, 2, 3], [5 * P, 3 * P], P=P, fp8=fp8, seed=P).check()


@pytest.mark.parametrize("T", [2, 3, 5, 16])
@pytest.mark.parametrize("fp8,kvs", [(False, False), (False, True), (True, False)])
def test_query_tokens(T, fp8, kvs):
    Case(16, 4, 512, [T, T + 1, 50, 17 + T], [0, 1, 4], [272, 160], T=T, fp8=fp8, kvs=kvs, seed=T).check()


def test_groups_of_every_kind():
    """Empty groups, groups of one, no prefix, no own tokens, nothing at all."""
    lens = [5, 0, 17, 0, 3, 0, 64]
    Case(16, 4, 512, lens, [0, 0, 1, 3, 3, 4, 6, 7], [160, 32, 0, 48, 0, 1008, 16], seed=3).check()
    c = Case(16, 4, 512, [0, 0], [0, 2], [0], seed=3)
    out = c.check()
    assert not out.view(torch.int16).any()


def test_many_groups():
    rng = random.Random(2)
    lens = [rng.randint(1, 20) for _ in range(80)]
    starts = [0] + sorted(rng.sample(range(1, 80), 39)) + [80]
    Case(8, 2, 512, lens, starts, [16 * rng.randint(0, 30) for _ in range(40)], seed=8).check()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("q_std", [0.0, 0.01, 12.0])
def test_score_ranges(q_std, fp8):
    """Flat softmaxes, and peaked ones whose running maximum keeps moving."""
    Case(16, 4, 512, [9, 70], [0, 2], [3008], q_std=q_std, fp8=fp8, seed=4).check()


def test_rising_scores():
    """Scores that rise along the prefix by hundreds: every tile moves the maximum."""
    c = Case(16, 4, 512, [20, 3], [0, 2], [2560], seed=6)
    idx = torch.tensor(c.ptab[0], device="cuda")
    ramp = torch.arange(2560, device="cuda").view(160, 1, 16, 1) / 2560 * 40
    c.kp[idx] = (c.q[0, 0].float().sign() * ramp).to(torch.bfloat16)
    c.check()


def test_plan_for_longer_lengths_serves_shorter_ones():
    c = Case(16, 4, 512, [5, 30, 2], [0, 2, 3], [160, 480], seed=1)
    c.check(c.step(lens=[32, 32, 32], prefix_lens=[480, 480]))
    c.check(c.step(lens=[1, 1, 1], prefix_lens=[0, 16]))  # longer than planned: the last piece takes the rest


def test_same_bits_on_every_run_and_in_any_company():
    """No order of arrival in the sums; and a row's result does not depend on its tile's other rows."""
    c = Case(16, 4, 512, [5, 30, 2, 8], [0, 4], [4000], seed=1)
    step = c.step()
    a, _ = c.run(step)
    for _ in range(3):
        o, _ = c.run(step)
        assert torch.equal(a.view(torch.int16), o.view(torch.int16))
    c.q[1] *= 9
    o, _ = c.run(step)
    keep = [0, 2, 3]
    assert torch.equal(a[keep].view(torch.int16), o[keep].view(torch.int16))


@pytest.mark.parametrize("batch", [2, 7, 15, 40])
@pytest.mark.parametrize("fp8", [False, True])
def test_many_runs_give_the_same_bits(batch, fp8):
    # calls in a row, each overlapping the ends of the others: what one stage of a ring
    # took from the wrong copy would show as a run that differs
    c = Case(16, 4, 512, [20] * batch, [0, batch], [8000], fp8=fp8, seed=batch)
    ref, step = c.run()
    outs = [torch.empty_like(ref) for _ in range(200)]
    for o in outs:
        c.run(step, o)
    assert step.check() == 0
    assert all(torch.equal(o.view(torch.int16), ref.view(torch.int16)) for o in outs)


def test_agrees_with_plain_decode():
    """One table per request over the same pages: decode's result, within both tolerances."""
    c = Case(16, 4, 512, [17, 64, 1], [0, 3], [608], seed=2, garbage=False)
    out = c.check()
    table = torch.cat([c.dev["ptab"].expand(3, -1), c.dev["table"]], 1).contiguous()
    lens = [608 + n for n in c.lens]
    step = b.LayerStep(16, 4, 512, 16, c.pages, table.shape[1], lens)
    ref = step(c.q, c.kp, c.vp, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), c.scale,
               torch.empty_like(c.q))
    _, tol = c.expect()
    assert ((out.double() - ref.double()).abs() <= 2 * tol).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_bad_prefix_pages_are_masked_and_flagged(fp8):
    c = Case(16, 4, 512, [9, 40], [0, 2], [480], fp8=fp8, seed=5)
    bad = c.dev["ptab"].clone()
    bad[0, [3, 29]] = torch.tensor([-1, c.pages], dtype=torch.int32, device="cuda")
    good = [p for i, p in enumerate(c.ptab[0]) if i not in (3, 29)]
    c.dev["ptab"] = bad
    out, step = c.run()
    with pytest.raises(b.PagedDecodeError) as e:
        step.check()
    assert e.value.flags == b.PD_DEVFLAG_BAD_PAGE
    c.ptab, c.prefix = [good], [448]
    exp, tol = c.expect()
    assert ((out.double() - exp).abs() <= tol).all()


def test_every_prefix_page_bad():
    c = Case(16, 4, 512, [9, 40], [0, 2], [480], seed=5)
    c.dev["ptab"].fill_(c.pages + 7)
    out, step = c.run()
    with pytest.raises(b.PagedDecodeError) as e:
        step.check()
    assert e.value.flags == b.PD_DEVFLAG_BAD_PAGE
    c.ptab, c.prefix = [[]], [0]
    exp, tol = c.expect()
    assert ((out.double() - exp).abs() <= tol).all()


@pytest.mark.parametrize("plen,used", [(-16, 0), (10 ** 6, 480), (479, 464)])
def test_bad_prefix_length_is_cut_and_flagged(plen, used):
    c = Case(16, 4, 512, [9, 40], [0, 2], [480], seed=5)
    step = c.step()
    c.dev["plens"][0] = plen
    out, _ = c.run(step)
    with pytest.raises(b.PagedDecodeError) as e:
        step.check()
    assert e.value.flags == b.PD_DEVFLAG_BAD_SEQLEN
    c.prefix = [used]
    exp, tol = c.expect()
    assert ((out.double() - exp).abs() <= tol).all()


@pytest.mark.parametrize("starts", [[1, 2, 4], [0, 5, 4], [0, 2, 3], [0, -3, 4], [0, 2, 99]])
def test_bad_group_starts_are_flagged(starts):
    c = Case(16, 4, 512, [9, 40, 3, 3], [0, 2, 4], [480, 16], seed=5)
    step = c.step()
    c.dev["starts"].copy_(torch.tensor(starts, dtype=torch.int32))
    c.run(step)
    with pytest.raises(b.PagedDecodeError) as e:
        step.check()
    assert e.value.flags & b.PD_DEVFLAG_BAD_GROUP


def test_more_row_tiles_than_planned_are_flagged():
    c = Case(16, 4, 512, [3] * 32, [0, 32, 32, 32], [480, 16, 16], seed=5)
    step = c.step()
    c.dev["starts"].copy_(torch.tensor([0, 1, 2, 32], dtype=torch.int32))
    c.run(step)
    with pytest.raises(b.PagedDecodeError) as e:
        step.check()
    assert e.value.flags & b.PD_DEVFLAG_BAD_GROUP


def test_infinite_and_nan_rows_stay_their_own():
    """A NaN query gives NaN in its own row only."""
    c = Case(16, 4, 512, [9, 40, 8], [0, 3], [480], seed=5)
    a = c.check()
    c.q[1, 3] = float("nan")
    out, _ = c.run()
    assert out[1, 3].isnan().all()
    out[1, 3] = a[1, 3]
    assert torch.equal(out.view(torch.int16), a.view(torch.int16))


def test_captured_and_on_another_stream():
    c = Case(16, 4, 512, [9, 40, 8], [0, 3], [1600], seed=5)
    step = c.step()
    a = c.check(step)
    s = torch.cuda.Stream()
    out = torch.zeros_like(c.q)
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c.run(step, out)
        s.synchronize()
        assert torch.equal(out, a)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            c.run(step, out)
    c.q.copy_(torch.randn_like(c.q.float()))
    torch.cuda.synchronize()
    g.replay()
    torch.cuda.synchronize()
    e, tol = c.expect()
    assert ((out.double() - e).abs() <= tol).all()


def test_long_prefix_past_32_bit_offsets():
    """Pages at byte offsets past 2^32 of the pool."""
    P, H, d = 16, 4, 512
    pages = (1 << 32) // (P * H * d * 2) + 40
    g = torch.Generator(device="cuda").manual_seed(1)
    c = Case(16, 4, 512, [9, 30], [0, 2], [320], seed=5, kvs=True, garbage=False)
    big = torch.zeros(pages, H, P, d, dtype=torch.bfloat16, device="cuda")
    big[-c.pages:] = torch.randn(c.pages, H, P, d, generator=g, device="cuda").to(torch.bfloat16)
    c.kp = big
    move = lambda t: [[p + pages - c.pages if p >= 0 else p for p in r] for r in t]  # noqa: E731
    c.ptab, c.table = move(c.ptab), move(c.table)
    c.dev["ptab"] = torch.tensor(c.ptab, dtype=torch.int32, device="cuda")
    c.dev["table"] = torch.tensor(c.table, dtype=torch.int32, device="cuda")
    c.pages = pages
    c.check()


@pytest.mark.parametrize("Hq,Hkv,d,T", [(16, 4, 512, 1), (16, 4, 512, 4), (32, 2, 512, 1), (16, 8, 256, 5)])
@pytest.mark.parametrize("fp8,kvs", [(False, False), (False, True), (True, False), (True, True)])
def test_long_own_parts(Hq, Hkv, d, T, fp8, kvs):
    # own tokens in several pieces, and two column tiles in a CTA (no sum is longer than a piece's)
    Case(Hq, Hkv, d, [4200, 37, 1500], [0, 3], [64], T=T, fp8=fp8, kvs=kvs, seed=T).check()


@pytest.mark.parametrize("seed", range(24))
def test_random_shapes(seed):
    rng = random.Random(seed)
    Hq, Hkv, d = rng.choice(LAYERS)
    T = rng.choice((1, 1, 2, 4)) if d > 128 else 1
    B = rng.choice((1, 2, 7, 20, 45))
    N = rng.randint(1, min(B, 4))
    P = rng.choice((16, 32, 48, 64))
    starts = [0] + sorted(rng.randint(0, B) for _ in range(N - 1)) + [B]
    Case(Hq, Hkv, d, [rng.randint(T, 150) for _ in range(B)], starts,
         [P * rng.randint(0, 2000 // P) for _ in range(N)], T=T, P=P, kvs=rng.random() < 0.4,
         fp8=d > 128 and rng.random() < 0.4, seed=seed, q_std=rng.choice((0.5, 1.0, 3.0))).check()


@pytest.mark.parametrize("kvs", [False, True])
@pytest.mark.parametrize("code", [1, 7, 8, 0x78, 0x7e, 0x81, 0xfe])
def test_fp8_codes(code, kvs):
    """Subnormal, smallest normal and largest e4m3 codes, both signs: V of one
    code everywhere gives that code's value times its scale."""
    c = Case(16, 4, 512, [9, 30], [0, 2], [272], fp8=True, kvs=kvs, seed=1, garbage=False)
    (c.kp if kvs else c.vp).fill_(code)
    scale = c.ks if kvs else c.vs
    scale.copy_(torch.full_like(scale, 0.013))
    c.check()


def test_fp8_scales_of_very_different_pages():
    """Page scales over six orders of magnitude, K's and V's each its own."""
    c = Case(16, 4, 512, [40, 3], [0, 2], [1600], fp8=True, seed=1)
    g = torch.Generator(device="cuda").manual_seed(7)
    c.vs *= 10.0 ** (torch.rand(c.vs.shape, generator=g, device="cuda") * 6 - 3)
    c.ks *= torch.rand(c.ks.shape, generator=g, device="cuda") * 1.5 + 0.25
    c.check()


@pytest.mark.parametrize("batch,fp8", [(3, False), (40, False), (40, True)])
@pytest.mark.parametrize("jump", [20.0, 200.0, 3000.0])
def test_scores_that_jump_far_past_the_first_tile(batch, fp8, jump):
    """One later token's score is far above all before it: past the references'
    range, and past what an exponential can hold."""
    c = Case(16, 4, 512, [7] * batch, [0, batch], [1200], fp8=fp8, seed=9, q_std=1.0, garbage=False)
    at = 900
    page = c.ptab[0][at // 16]
    q = c.q.view(batch, 4, 4, 512)
    c.q.copy_(q[:, :, :1].expand_as(q).reshape(c.q.shape))  # one direction per KV head and request
    c.q[1:] = c.q[:1]
    direction = c.q.view(batch, 4, 4, 512)[0, :, 0].float()
    value = direction / direction.norm(dim=1, keepdim=True) * (jump * 22.6 / direction.norm(dim=1, keepdim=True))
    if fp8:
        big = value.abs().amax(1)
        c.ks[page] = torch.maximum(c.ks[page], big / 448)
        rows = c.kp[page].view(torch.float8_e4m3fn).float() * 0
        rows[:, at % 16] = value / c.ks[page][:, None]
        c.kp[page] = rows.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        c.kp[page, :, at % 16] = value.to(torch.bfloat16)
    c.check()


def test_infinite_scores():
    """An infinite cached key gives its softmax's NaN to the rows that see it, and to no other KV head's."""
    c = Case(16, 4, 512, [9, 30], [0, 2], [640], seed=3)
    a = c.check()
    c.kp[c.ptab[0][10], 2, 5] = float("inf")
    out, _ = c.run()
    assert out[:, 8:12].isnan().all()
    keep = [h for h in range(16) if not 8 <= h < 12]
    assert torch.equal(out[:, keep], a[:, keep])


def test_negative_and_zero_scale():
    for scale in (-0.05, 0.0):
        c = Case(16, 4, 512, [9, 30], [0, 2], [640], seed=3)
        c.scale = scale
        c.check()
