"""Decode attention over a 4-bit cache against a plain statement in 64 bits.

Tolerance, per output element, from the kernel's roundings:
  - a query element enters as 4-bit terms that leave out at most 0.177^6 = 3.1e-5 of the largest q of its 16 dims (plus
    2^-18 of the row's largest, where the last scales are e4m3's smallest), so a score is off by at most
    scale * sum_blocks (3.1e-5 max|q| + 2^-18 max|q_row|) sum|k|, and by fp32 sums of 512 products (2^-14 of sum|q k|
    at most, far less in fact: 512 roundings of 2^-24);
  - probabilities are rounded to tf32: by 2^-11 of themselves; below 2^-126 of their reference, which is at most 2^60
    below the largest, they may vanish, which 2^-40 of the largest weight (at most 1) per token covers; exponentials are
    within 2^-21;
  - the output is rounded to bf16 (2^-8).
With e = the largest score error of a row and w the exact weights, weights are off by a factor of at most
exp(2 e) (1 + 2^-10) and by 2^-40, so |out - exact| <= 2^-8 |exact| + (exp(2 e) (1 + 2^-10) - 1) * 2 * sum w |v| +
2^-40 * sum |v| over the tokens.
"""
import math

import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b

pytestmark = pytest.mark.gpu

E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def values(codes, scales, exp):
    """What codes [..., d / 2] under e4m3 scales [..., d / 16] stand for, in 64 bits."""
    lut = torch.tensor(E2M1 + [-x for x in E2M1], dtype=torch.float64, device=codes.device)
    x = lut[torch.stack([codes & 15, codes >> 4], -1).flatten(-2).long()]
    s = scales.view(torch.float8_e4m3fn).double() * 2.0 ** exp
    return x * s.repeat_interleave(16, -1)


def random_pool(pages, heads, P, d, g, spread=1.0):
    codes = torch.randint(0, 256, (pages, heads, P, d // 2), generator=g, device="cuda", dtype=torch.uint8)
    s = torch.exp(torch.randn((pages, heads, P, d // 16), generator=g, device="cuda") * spread) * 0.5
    return codes, s.clamp(2.0 ** -9, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


class Case:
    def __init__(self, Hq, Hkv, d, lens, T=1, P=16, window=0, kvs=False, k_exp=0, v_exp=0, seed=0, q_std=1.0, spread=0.5):
        g = torch.Generator(device="cuda").manual_seed(seed)
        cg = torch.Generator().manual_seed(seed)
        self.T, self.P, self.window, self.kvs, self.k_exp, self.v_exp = T, P, window, kvs, k_exp, k_exp if kvs else v_exp
        self.Hq, self.Hkv, self.d, self.lens_list = Hq, Hkv, d, list(lens)
        B = len(lens)
        held = [-(-n // P) for n in lens]
        self.pages, self.width = sum(held) + 3, max(1, max(held) + 1)
        perm = torch.randperm(self.pages, generator=cg).tolist()
        table = torch.full((B, self.width), -1, dtype=torch.int32)
        at = 0
        for i, n in enumerate(held):
            table[i, :n] = torch.tensor(perm[at:at + n], dtype=torch.int32)
            at += n
        self.table, self.lens = table.cuda(), torch.tensor(list(lens), dtype=torch.int32).cuda()
        self.kc, self.ks = random_pool(self.pages, Hkv, P, d, g, spread)
        self.vc, self.vs = (None, None) if kvs else random_pool(self.pages, Hkv, P, d, g, spread)
        self.q = (torch.randn((B, T, Hq, d), generator=g, device="cuda") * q_std * 2.0 ** -k_exp / math.sqrt(16)).to(
            torch.bfloat16)
        self.scale = 1.0 / math.sqrt(d)

    def step(self, **kw):
        return b.LayerStep(self.Hq, self.Hkv, self.d, self.P, self.pages, self.width, kw.pop("plan_lens", self.lens_list),
                           window=self.window, kv_shared=self.kvs, kv_dtype=b.PD_KV_FP4_E2M1, query_tokens=self.T, **kw)

    def run(self, step=None, out=None, check=True):
        step = step or self.step()
        q = self.q if self.T > 1 else self.q[:, 0]
        out = torch.full_like(q, 7.0) if out is None else out
        step(q, self.kc, self.vc, self.table, self.lens, self.scale, out, k_scale=self.ks, v_scale=self.vs,
             k_exp=self.k_exp, v_exp=self.v_exp)
        if check:
            step.check()
        return out.view(self.q.shape)

    def rows(self, codes, scales, i, n, exp):
        pages = self.table[i].long()[: -(-n // self.P)]
        x = values(codes[pages], scales[pages], exp)  # [pages, H, P, d]
        return x.transpose(1, 2).reshape(-1, self.Hkv, self.d)[:n]

    def exact(self):
        """(exact output, its tolerance), [B, T, Hq, d] in 64 bits."""
        out = torch.zeros(self.q.shape, dtype=torch.float64, device="cuda")
        tol = torch.zeros_like(out)
        for i, n in enumerate(self.lens.tolist()):
            if n == 0:
                continue
            k = self.rows(self.kc, self.ks, i, n, self.k_exp)
            v = k if self.kvs else self.rows(self.vc, self.vs, i, n, self.v_exp)
            q = self.q[i].double().view(self.T, self.Hkv, -1, self.d)
            s = torch.einsum("thgd,nhd->thgn", q, k) * self.scale
            pos = torch.arange(n, device="cuda")
            last = n - self.T + torch.arange(self.T, device="cuda")[:, None]
            seen = (pos <= last) & ((pos > last - self.window) if self.window else (pos >= 0))
            seen = seen[:, None, None]
            # the score's error, block by block
            qa = q.abs().unflatten(-1, (-1, 16)).amax(-1)
            lost = 3.1e-5 * qa + 2.0 ** -18 * qa.amax(-1, keepdim=True)
            ka = k.abs().unflatten(-1, (-1, 16)).sum(-1)
            err = torch.einsum("thgb,nhb->thgn", lost, ka) + 512 * 2.0 ** -24 * torch.einsum(
                "thgd,nhd->thgn", q.abs(), k.abs())
            e = (err * abs(self.scale)).masked_fill(~seen, 0).amax(-1, keepdim=True)  # |scale x| errs by |scale| |error of x|
            w = torch.softmax(s.masked_fill(~seen, -math.inf), -1)
            w = torch.nan_to_num(w, nan=0.0)  # a token that attends nothing
            o = torch.einsum("thgn,nhd->thgd", w, v)
            mag = torch.einsum("thgn,nhd->thgd", w, v.abs())
            out[i] = o.reshape(self.T, self.Hq, self.d)
            tail = 2.0 ** -40 * v.abs().sum(0).repeat_interleave(self.Hq // self.Hkv, 0).view(self.Hkv, -1, self.d)
            t = 2.0 ** -8 * o.abs() + (torch.exp(2 * e) * (1 + 2.0 ** -10) - 1) * 2 * mag + tail
            tol[i] = t.reshape(self.T, self.Hq, self.d)
        return out, tol


def compare(c, got):
    want, tol = c.exact()
    over = (got.double() - want).abs() - tol
    assert torch.isfinite(got.float()).all()
    assert float(over.max()) <= 0, f"off by {float(over.max()):.3g} past the tolerance at {int(over.argmax())}"


@pytest.mark.parametrize("lens", [[1], [16], [17], [127, 128, 129], [0, 300, 1], [1000], [5, 2049, 64, 700]])
@pytest.mark.parametrize("Hq,Hkv,d", [(16, 4, 512), (8, 8, 256)])
@pytest.mark.parametrize("kvs", [False, True])
def test_lengths(lens, Hq, Hkv, d, kvs):
    c = Case(Hq, Hkv, d, lens, kvs=kvs, seed=len(lens))
    compare(c, c.run())


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 6, 7, 8, 9, 12, 16])
@pytest.mark.parametrize("d", [256, 512])
def test_groups(group, d):
    c = Case(2 * group, 2, d, [333, 90], seed=group)
    compare(c, c.run())


@pytest.mark.parametrize("T", [2, 3, 5, 17])
@pytest.mark.parametrize("Hq,Hkv,d,window", [(16, 4, 512, 0), (24, 4, 512, 0), (16, 8, 256, 0), (16, 8, 256, 100),
                                             (32, 4, 256, 33)])
@pytest.mark.parametrize("kvs", [False, True])
def test_query_tokens(T, Hq, Hkv, d, window, kvs):
    c = Case(Hq, Hkv, d, [T, 150, 129 + T, 1025], T=T, window=window, kvs=kvs, seed=T)
    compare(c, c.run())


@pytest.mark.parametrize("window", [1, 15, 16, 100, 1000, 1024])
@pytest.mark.parametrize("Hq,Hkv,d", [(16, 8, 256), (16, 4, 512)])
def test_windows(window, Hq, Hkv, d):
    c = Case(Hq, Hkv, d, [1, 99, 1500, 2777], window=window, seed=window)
    compare(c, c.run())


@pytest.mark.parametrize("P", [16, 32, 48, 64, 128, 256])
def test_page_sizes(P):
    c = Case(16, 4, 512, [700, 33, 1], P=P, seed=P)
    compare(c, c.run())


@pytest.mark.parametrize("k_exp,v_exp", [(-64, 64), (64, -64), (-7, 3), (5, -9)])
@pytest.mark.parametrize("kvs", [False, True])
def test_exponents(k_exp, v_exp, kvs):
    c = Case(8, 2, 256, [500, 77], k_exp=k_exp, v_exp=v_exp, kvs=kvs, seed=1)
    compare(c, c.run())


@pytest.mark.parametrize("lens", [[20000], [9000, 40000], [3000] * 8, [600] * 40, [100] * 200])
@pytest.mark.parametrize("Hq,Hkv,d,kvs", [(16, 4, 512, False), (16, 4, 512, True), (16, 8, 256, False)])
def test_pieces(lens, Hq, Hkv, d, kvs):
    """Pieces merged by a launch of their own, in a cluster, and none."""
    c = Case(Hq, Hkv, d, lens, kvs=kvs, seed=7)
    compare(c, c.run())


@pytest.mark.parametrize("sms", [1, 8, 37, 152, 300])
def test_piece_counts(sms):
    c = Case(8, 2, 512, [1111, 640, 128], seed=sms)
    compare(c, c.run(c.step(sm_count=sms)))


@pytest.mark.parametrize("q_std", [1e-30, 1e-3, 8.0, 60.0])
def test_query_magnitudes(q_std):
    c = Case(16, 4, 512, [700, 40], q_std=q_std, spread=0.2, seed=3)
    compare(c, c.run())


def test_one_channel_large():
    """A query channel far above the others, which then have scales near e4m3's smallest."""
    c = Case(16, 4, 512, [700, 40], seed=4)
    c.q[..., 100] *= 300
    compare(c, c.run())


def test_zero_query_and_zero_rows():
    c = Case(16, 4, 512, [260], seed=5)
    c.q[:, :, 3] = 0
    c.vs[:] = 0
    got = c.run()
    assert not got.any()
    c = Case(16, 4, 512, [260], seed=5)
    c.q[:, :, 3] = 0
    compare(c, c.run())


def test_nan_and_infinity_in_a_query_row_stay_there():
    c = Case(16, 4, 512, [700, 40], seed=6)
    clean = c.run()
    c.q[0, 0, 2, 5], c.q[1, 0, 9, 500] = math.nan, math.inf
    got = c.run()
    assert got[0, 0, 2].isnan().all() and got[1, 0, 9].isnan().all()
    keep = torch.ones(2, 16, dtype=torch.bool, device="cuda")
    keep[0, 2] = keep[1, 9] = False
    assert torch.equal(got[:, 0][keep], clean[:, 0][keep])


@pytest.mark.parametrize("kvs", [False, True])
def test_nan_in_unattended_rows(kvs):
    """Rows behind the length, in front of the window and in pages nobody holds may hold any bits."""
    c = Case(16, 8, 256, [700, 41, 0], window=300, kvs=kvs, seed=8)
    clean = c.run()
    used = torch.zeros((c.pages, c.P), dtype=torch.bool, device="cuda")
    for i, n in enumerate(c.lens_list):
        for t in range(max(0, n - 300), n):
            used[int(c.table[i, t // c.P]), t % c.P] = True
    for s in (c.ks, c.vs):
        if s is not None:
            s.transpose(1, 2)[~used] = 0x7F
    assert torch.equal(c.run(), clean)


def test_nan_row_attended():
    c = Case(16, 4, 512, [400], seed=9)
    page, off = int(c.table[0, 3]), 5
    c.ks[page, 1, off, 7] = 0x7F
    got = c.run()
    assert got[0, 0, 4:8].isnan().all() and torch.isfinite(got[0, 0, :4].float()).all()
    c = Case(16, 4, 512, [400], seed=9)
    c.vs[page, 2, off, 7] = 0x7F
    got = c.run()
    assert got[0, 0, 8:12, 112:128].isnan().all()
    bad = got.isnan()
    bad[0, 0, 8:12, 112:128] = False
    assert not bad.any()


@pytest.mark.parametrize("window", [0, 40])
def test_nan_row_of_a_later_token(window):
    """A NaN in a new token's V row reaches the query tokens that attend it, and no earlier one; in front of a window
    likewise no later one."""
    T, n = 4, 200
    c = Case(16, 8, 256, [n], T=T, window=window, seed=10)
    clean = c.run()
    for pos in (n - 2, n - T - 38) if window else (n - 2,):
        c = Case(16, 8, 256, [n], T=T, window=window, seed=10)
        c.vs[int(c.table[0, pos // 16]), 3, pos % 16, 2] = 0x7F
        got = c.run()
        for j in range(T):
            last = n - T + j
            attends = pos <= last and (not window or pos > last - window)
            assert got[0, j, 6:8, 32:48].isnan().all() == attends, (pos, j)
            rest = got[0, j].isnan()
            rest[6:8, 32:48] = False
            assert not rest.any()
            if not attends:
                assert torch.equal(got[0, j], clean[0, j])


def test_bad_page_is_masked_and_reported():
    c = Case(16, 4, 512, [700], seed=11)
    for bad in (-1, c.pages, 2 ** 30):
        c.table[0, 5] = bad
        step = c.step()
        got = c.run(step, check=False)
        with pytest.raises(b.PagedDecodeError) as e:
            step.check()
        assert e.value.flags == b.PD_DEVFLAG_BAD_PAGE
        assert torch.isfinite(got.float()).all()
        assert step.check() == 0
        # as if those 16 tokens were not there
        o = Case(16, 4, 512, [700], seed=11)
        keep = torch.cat([torch.arange(80), torch.arange(96, 700)]).cuda()
        k, v = o.rows(o.kc, o.ks, 0, 700, 0)[keep], o.rows(o.vc, o.vs, 0, 700, 0)[keep]
        w = torch.softmax(torch.einsum("hgd,nhd->hgn", o.q[0, 0].double().view(4, 4, 512), k) * o.scale, -1)
        want = torch.einsum("hgn,nhd->hgd", w, v).reshape(16, 512)
        assert float((got[0, 0].double() - want).norm() / want.norm()) < 2.0 ** -7


def test_bad_length_is_cut_and_reported():
    c = Case(16, 4, 512, [320], seed=12)
    step = c.step()
    c.lens[0] = c.width * 16 + 5
    c.table[0] = torch.where(c.table[0] < 0, 0, c.table[0])
    got = c.run(step, check=False)
    with pytest.raises(b.PagedDecodeError) as e:
        step.check()
    assert e.value.flags == b.PD_DEVFLAG_BAD_SEQLEN
    c.lens[0] = c.width * 16
    assert torch.equal(got, c.run(step))
    c.lens[0] = -3
    assert not c.run(step, check=False).any()
    with pytest.raises(b.PagedDecodeError):
        step.check()


def test_longer_lengths_than_planned_and_shorter():
    c = Case(16, 4, 512, [1500, 1400], seed=13)
    step = c.step(plan_lens=[1500, 1500])
    compare(c, c.run(step))
    c.lens = torch.tensor([3, 1399], dtype=torch.int32, device="cuda")
    compare(c, c.run(step))


def test_a_stalled_copy_gives_up():
    c = Case(16, 4, 512, [700], seed=14)
    step = c.step()
    good = c.run(step)
    step.plan.test_stall_bytes = 16
    c.run(step, check=False)
    with pytest.raises(b.PagedDecodeError) as e:
        step.check()
    assert e.value.flags & b.PD_DEVFLAG_WAIT_TIMEOUT
    step.plan.test_stall_bytes = 0
    assert torch.equal(c.run(step), good)


@pytest.mark.parametrize("lens,kvs", [([32768] * 4, False), ([5000, 100, 20000], True), ([1024] * 8, False)])
def test_same_bits_every_run(lens, kvs):
    c = Case(16, 4, 512, lens, kvs=kvs, seed=15)
    step = c.step()
    first = c.run(step)
    for _ in range(50):
        assert torch.equal(c.run(step, check=False), first)
    step.check()


def test_captured_and_replayed_over_changing_inputs():
    c, o = Case(16, 4, 512, [1024] * 8, seed=16), Case(16, 4, 512, [1024] * 8, seed=17)
    step = c.step()
    out = torch.empty_like(c.q[:, 0])
    c.run(step, out=out)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(step, out=out, check=False)
    for x in (o, Case(16, 4, 512, [1024] * 8, seed=18)):
        for name in ("q", "kc", "ks", "vc", "vs", "table", "lens"):
            getattr(c, name).copy_(getattr(x, name))
        out.fill_(3.0)
        graph.replay()
        step.check()
        assert torch.equal(out, x.run()[:, 0])


def test_on_another_stream():
    c = Case(16, 4, 512, [3000, 500], seed=19)
    want = c.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    step = c.step()
    torch.cuda.current_stream().synchronize()
    with torch.cuda.stream(s):
        got = c.run(step)
    assert torch.equal(got, want)


@pytest.mark.parametrize("T", [1, 3])
def test_early_copies(T):
    """With early_kv, behind a launch that writes each request's newest rows."""
    c = Case(16, 4, 512, [900, 33, 128 + T], T=T, seed=20)
    desc = b.layer_desc(16, 4, 512, 16, c.pages, c.width, kv_dtype=b.PD_KV_FP4_E2M1)
    pos = [(i, n - T + j) for i, n in enumerate(c.lens_list) for j in range(T)]
    slots = torch.tensor([int(c.table[i, t // 16]) * 16 + t % 16 for i, t in pos], dtype=torch.int32, device="cuda")
    k = torch.empty((len(pos), 4, 512), dtype=torch.bfloat16, device="cuda")
    v = torch.empty_like(k)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.paged_decode_read_slots_fp4(desc, slots, c.kc, c.vc, c.ks, c.vs, k, v, flags)
    b.paged_decode_write_slots_fp4(desc, k, v, slots, c.kc, c.vc, c.ks, c.vs, flags)
    want = c.run()  # (the rows as they are quantised again)
    step = c.step(early_kv=True)
    for _ in range(20):
        b.paged_decode_write_slots_fp4(desc, k * 0, v * 0, slots, c.kc, c.vc, c.ks, c.vs, flags)
        b.paged_decode_write_slots_fp4(desc, k, v, slots, c.kc, c.vc, c.ks, c.vs, flags)
        assert torch.equal(c.run(step, check=False), want)
    step.check()
    assert int(flags) == 0
