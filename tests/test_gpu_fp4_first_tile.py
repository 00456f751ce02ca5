"""A 4-bit decode's first tile, right behind other work on the same SMs: the unit
matrix and its scales have to be in place before the first product that takes
them, however early the first tile has landed and whatever tensor memory held
before. Against the plain statement in 64 bits and the tolerance of
test_gpu_fp4.py."""
import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b
from test_gpu_fp4 import Case, compare
from test_gpu_shared import Case as SharedCase

pytestmark = pytest.mark.gpu

# (Hq, Hkv, d, T, window): 4 columns a CTA, and 8, of either head dim
LAYERS = [(16, 8, 256, 1, 0), (16, 8, 256, 1, 100), (32, 4, 256, 1, 0), (16, 4, 512, 1, 0), (16, 4, 512, 2, 0),
          (24, 4, 512, 1, 0)]


def newest_rows(c):
    """(layer, slots, k, v) of a write that leaves the newest rows of every request as they are."""
    desc = b.layer_desc(c.Hq, c.Hkv, c.d, c.P, c.pages, c.width, c.window, c.kvs, b.PD_KV_FP4_E2M1)
    pos = [(i, n - c.T + j) for i, n in enumerate(c.lens_list) for j in range(c.T)]
    slots = torch.tensor([int(c.table[i, t // c.P]) * c.P + t % c.P for i, t in pos], dtype=torch.int32, device="cuda")
    k = torch.empty((len(pos), c.Hkv, c.d), dtype=torch.bfloat16, device="cuda")
    v = None if c.kvs else torch.empty_like(k)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    pools = (c.kc, c.vc, c.ks, c.vs)
    b.paged_decode_read_slots_fp4(desc, slots, *pools, k, v, flags)
    b.paged_decode_write_slots_fp4(desc, k, v, slots, *pools, flags)  # (as they are quantised again)
    return desc, slots, k, v, flags


@pytest.mark.parametrize("early", [False, True])
@pytest.mark.parametrize("kvs", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,T,window", LAYERS)
def test_behind_a_prefix_pass(Hq, Hkv, d, T, window, kvs, early):
    """The prefix pass writes tensor memory; the cache write follows it, then the decode."""
    c = Case(Hq, Hkv, d, [900, 33, 128 + T, 2000], T=T, window=window, kvs=kvs, seed=T + d)
    desc, slots, k, v, flags = newest_rows(c)
    want, tol = c.exact()
    other = SharedCase(16, 4, 512, [100] * 20, [0, 20], [2000], seed=5)
    prefix, step = other.step(), c.step(early_kv=early)
    got, theirs = [], torch.empty_like(other.q)
    for _ in range(10):
        other.run(prefix, theirs)
        b.paged_decode_write_slots_fp4(desc, k, v, slots, c.kc, c.vc, c.ks, c.vs, flags)
        got.append(c.run(step, check=False))
    step.check()
    assert prefix.check() == 0 and int(flags) == 0
    for out in got:
        assert torch.isfinite(out.float()).all()
        assert float(((out.double() - want).abs() - tol).max()) <= 0
        assert torch.equal(out, got[0])


@pytest.mark.parametrize("kvs", [False, True])
@pytest.mark.parametrize("Hq,Hkv,d,T,window", LAYERS)
def test_early_copies_of_every_kind(Hq, Hkv, d, T, window, kvs):
    c = Case(Hq, Hkv, d, [900, 33, 128 + T, 2000], T=T, window=window, kvs=kvs, seed=3 * T + d)
    desc, slots, k, v, flags = newest_rows(c)
    want, tol = c.exact()
    step = c.step(early_kv=True)
    for _ in range(5):
        b.paged_decode_write_slots_fp4(desc, k, v, slots, c.kc, c.vc, c.ks, c.vs, flags)
        out = c.run(step, check=False)
        assert float(((out.double() - want).abs() - tol).max()) <= 0
    step.check()
    assert int(flags) == 0


@pytest.mark.parametrize("sms", [1, 152])
def test_behind_a_prefix_pass_in_a_graph(sms):
    c = Case(16, 8, 256, [700, 40, 1500], window=300, seed=8)
    other = SharedCase(16, 8, 256, [64] * 12, [0, 5, 12], [1024, 512], seed=6)
    step, prefix = c.step(sm_count=sms), other.step()
    out, theirs = torch.empty_like(c.q[:, 0]), torch.empty_like(other.q)

    def both():
        other.run(prefix, theirs)
        c.run(step, out=out, check=False)

    both()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        both()
    for _ in range(10):
        out.fill_(7.0)
        graph.replay()
        step.check()
        compare(c, out.view(c.q.shape))
