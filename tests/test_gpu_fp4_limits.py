"""Decode over a 4-bit cache at the ends of its ranges: the most query tokens and
heads, pools whose codes and scales pass 32-bit offsets, long contexts. Against
the plain statement in 64 bits and the tolerance of test_gpu_fp4.py."""
import pytest
import torch

from test_gpu_fp4 import Case, compare

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,Hq,Hkv,d,window,kvs", [(256, 32, 2, 512, 0, False), (256, 16, 1, 256, 33, True),
                                                   (255, 9, 1, 512, 0, True), (64, 16, 4, 512, 100, False),
                                                   (256, 4, 4, 256, 0, False)])
@pytest.mark.parametrize("sms", [5, 152])
def test_the_most_query_rows(T, Hq, Hkv, d, window, kvs, sms):
    c = Case(Hq, Hkv, d, [T, T + 1, 700, T + 129], T=T, window=window, kvs=kvs, seed=T + d)
    compare(c, c.run(c.step(sm_count=sms)))


@pytest.mark.parametrize("kvs", [False, True])
def test_pool_past_32_bit_offsets(kvs):
    # 2^27 rows and some: 2^32 bytes of scales, 2^35 of codes; the pages in use are the last ones
    c = Case(16, 4, 512, [700, 33, 2000], kvs=kvs, seed=1)
    want, tol = c.exact()
    small, c.pages = c.pages, (1 << 27) // (4 * 16) + 50
    for name in ("kc", "ks", "vc", "vs"):
        pool = getattr(c, name)
        if pool is not None:
            big = torch.empty((c.pages, *pool.shape[1:]), dtype=torch.uint8, device="cuda")
            big[-small:] = pool
            big[:small] = 0x7f  # what a wrapped offset would reach
            setattr(c, name, big)
    c.table = torch.where(c.table >= 0, c.table + (c.pages - small), c.table)
    got = c.run()
    assert float(((got.double() - want).abs() - tol).max()) <= 0


def test_a_long_context():
    c = Case(4, 1, 512, [131072, 1, 70001], seed=2)
    compare(c, c.run())
