"""Decode over a 4-bit cache where a CTA's share holds many units, few, or parts of
one; references that scores outgrow; graphs that share a workspace. The plain
statement and its tolerance are those of test_gpu_fp4.py."""
import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b
from test_gpu_fp4 import Case, compare, values

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("sms", [1, 2, 3, 5, 17, 151])
@pytest.mark.parametrize("Hq,Hkv,d,window,kvs", [(16, 4, 512, 0, False), (16, 4, 512, 0, True), (16, 8, 256, 100, False),
                                                 (8, 8, 256, 0, True)])
def test_units_of_one_share(sms, Hq, Hkv, d, window, kvs):
    # lengths of no tile, one, a few: shares begin and end anywhere in a unit
    c = Case(Hq, Hkv, d, [0, 700, 1, 128, 129, 0, 1300, 64, 257, 5], window=window, kvs=kvs, seed=sms)
    compare(c, c.run(c.step(sm_count=sms)))


@pytest.mark.parametrize("T,Hq,Hkv,d", [(3, 24, 4, 512), (20, 16, 4, 512), (7, 64, 4, 256)])
@pytest.mark.parametrize("sms", [2, 7])
def test_column_tiles_of_one_share(sms, T, Hq, Hkv, d):
    c = Case(Hq, Hkv, d, [T, 300, 129 + T, 40], T=T, seed=T)
    compare(c, c.run(c.step(sm_count=sms)))


@pytest.mark.parametrize("batch", [31, 32, 33, 65, 1100])
def test_many_requests(batch):
    # lengths are read 32 requests at a time
    c = Case(4, 1, 256, [(37 * i) % 90 for i in range(batch)], seed=batch)
    compare(c, c.run())
    compare(c, c.run(c.step(sm_count=3)))


def test_requests_without_tokens():
    c = Case(8, 2, 512, [0] * 40, seed=1)
    assert torch.equal(c.run(c.step(sm_count=4)), torch.zeros_like(c.q))


def grown(rise, sms, kvs, lens=(1000, 2000)):
    """Scores that rise by `rise` (in log2) from one run of 100 tokens to the next: q and K have one dim each that
    counts, V and the rest of K's dims little."""
    c = Case(4, 1, 512, list(lens), kvs=kvs, seed=int(rise) + sms)
    c.q.mul_(2.0 ** -20)
    c.q[..., 0] = 16.0
    c.kc[..., 0] = 0x02  # dim 0: 1.0, dim 1: 0
    pos = torch.zeros(c.pages, c.P, device="cuda")
    for i, n in enumerate(lens):
        at = torch.arange(-(-n // c.P) * c.P, device="cuda").view(-1, c.P)
        pos[c.table[i].long()[:at.shape[0]]] = (at // 100).float()
    c.ks[:, 0, :, 0] = (1 + pos).to(torch.float8_e4m3fn).view(torch.uint8)  # e4m3 holds 1..16, and even numbers to 32
    c.scale = rise / 16.0 * 0.6931471805599453
    return c


@pytest.mark.parametrize("kvs", [False, True])
@pytest.mark.parametrize("sms", [1, 2, 152])
@pytest.mark.parametrize("rise", [5.0, 40.0, 70.0, 200.0, -70.0])
def test_scores_that_outgrow_their_reference(rise, sms, kvs):
    # 70 and 200: the sums are rescaled at nearly every tile; 40: at every other; -70: never
    c = grown(rise, sms, kvs)
    compare(c, c.run(c.step(sm_count=sms)))


@pytest.mark.parametrize("kvs", [False, True])
def test_pieces_give_the_same_bits_every_run(kvs):
    c = Case(16, 4, 512, [4000, 33, 900, 0, 2500], kvs=kvs, seed=9)
    step = c.step()
    first = c.run(step).clone()
    for _ in range(20):
        assert torch.equal(c.run(step).view(torch.int16), first.view(torch.int16))


def test_two_graphs_share_a_workspace():
    a, z = Case(16, 4, 512, [3000, 500], seed=3), Case(16, 4, 512, [100, 1900], seed=4)
    # one plan and workspace serve both: the block tables' rows have to be as wide
    wide = max(a.width, z.width)
    for c in (a, z):
        table = torch.full((2, wide), -1, dtype=torch.int32, device="cuda")
        table[:, :c.width] = c.table
        c.table, c.width = table, wide
    pages = max(a.pages, z.pages)
    for c in (a, z):
        for n in ("kc", "ks", "vc", "vs"):
            p = getattr(c, n)
            setattr(c, n, torch.cat([p, p[:1].expand(pages - c.pages, *p.shape[1:])]).contiguous())
        c.pages = pages
    step = a.step(plan_lens=[3000, 1900])
    want = [c.run(step).clone() for c in (a, z)]
    graphs, outs = [], []
    for c in (a, z):
        out = torch.full_like(c.q[:, 0], 7.0)
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(step, out=out, check=False)
        graphs.append(g)
        outs.append(out)
    for _ in range(5):
        for g, out, w in zip(graphs, outs, want):
            out.fill_(9.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out.view(w.shape), w)
    step.check()


def test_counts_are_set_back_after_a_time_out():
    c = Case(16, 4, 512, [3000, 900], seed=5)
    step = c.step()
    want = c.run(step).clone()
    step.plan.test_stall_bytes = 16
    with pytest.raises(b.PagedDecodeError):
        c.run(step)
    step.plan.test_stall_bytes = 0
    head = step.workspace[:int(step.plan.lse_offset)]
    assert int(head.count_nonzero()) == 0
    for _ in range(3):
        assert torch.equal(c.run(step), want)
    assert int(head.count_nonzero()) == 0


@pytest.mark.parametrize("v_exp", [-64, 64])
def test_extreme_exponents_of_v(v_exp):
    # the results' exponent is applied last: over large sums of probabilities it would not be a normal number
    c = grown(59.0, 1, False, lens=(1500,))
    c.v_exp = v_exp
    got = c.run(c.step(sm_count=1))
    want, tol = c.exact()
    over = (got.double() - want).abs() - tol
    assert float(over.max()) <= 0
    assert float(values(c.vc, c.vs, v_exp).abs().max()) > 0


@pytest.mark.parametrize("T,window", [(1, 0), (3, 0), (3, 20)])
@pytest.mark.parametrize("sms", [1, 152])
def test_nan_block_of_a_shared_pool(T, window, sms):
    # as K it makes the whole output row NaN, of the query tokens that attend it and of no other
    c = Case(16, 4, 512, [500, 300], T=T, window=window, kvs=True, seed=T)
    step = c.step(sm_count=sms)
    clean = c.run(step).clone()
    at = 499 if T == 1 else 498  # attended by the tokens from position 498 on: not by the first of three
    page = int(c.table[0, at // c.P])
    c.ks[page, 2, at % c.P, 5] = 0x7f
    got = c.run(step)
    hit = torch.zeros(c.q.shape, dtype=torch.bool, device="cuda")
    hit[0, (0 if T == 1 else 1):, 8:12] = True
    assert torch.isnan(got[hit]).all()
    assert torch.equal(got[~hit], clean[~hit])


def test_two_streams_at_once():
    cases = [Case(16, 4, 512, [3000, 700], seed=21), Case(16, 8, 256, [900, 40, 2000], window=300, kvs=True, seed=22)]
    steps = [c.step() for c in cases]
    want = [c.run(s).clone() for c, s in zip(cases, steps)]
    outs = [[torch.full_like(c.q[:, 0], 7.0) for _ in range(20)] for c in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for i in range(20):
        for c, s, o, st in zip(cases, steps, outs, streams):
            with torch.cuda.stream(st):
                c.run(s, out=o[i], check=False)
    torch.cuda.synchronize()
    for s, o, w in zip(steps, outs, want):
        s.check()
        assert all(torch.equal(x.view(w.shape), w) for x in o)
