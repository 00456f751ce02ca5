"""Decode over a 4-bit cache with query rows whose channels lie far apart: what is
left out of a query element follows the largest of its 16 dims, not its row's.

The large channel's 16 dims have K = 0, so that the others decide the scores.
Tolerance: the query's terms leave out at most 2^-14 of the largest of 16 and 2^-27 of the row's largest; everything
else as in test_gpu_fp4.py (fp32 sums of d products, tf32 probabilities, the output's bf16)."""
import pytest
import torch

from test_gpu_fp4 import Case

pytestmark = pytest.mark.gpu


def exact(c):
    """(exact output, tolerance) [B, Hq, d] of one query token a request, in 64 bits."""
    outs, tols = [], []
    for i, n in enumerate(c.lens_list):
        k = c.rows(c.kc, c.ks, i, n, c.k_exp)
        v = k if c.kvs else c.rows(c.vc, c.vs, i, n, c.v_exp)
        q = c.q[i, 0].double().view(c.Hkv, -1, c.d)
        w = torch.softmax(torch.einsum("hgd,nhd->hgn", q, k) * c.scale, -1)
        qa = q.abs().unflatten(-1, (-1, 16)).amax(-1)
        lost = 2.0 ** -14 * qa + 2.0 ** -27 * qa.amax(-1, keepdim=True)
        err = torch.einsum("hgb,nhb->hgn", lost, k.abs().unflatten(-1, (-1, 16)).sum(-1))
        err = err + 512 * 2.0 ** -24 * torch.einsum("hgd,nhd->hgn", q.abs(), k.abs())
        e = (err * c.scale).amax(-1, keepdim=True)
        o, mag = torch.einsum("hgn,nhd->hgd", w, v), torch.einsum("hgn,nhd->hgd", w, v.abs())
        tail = 2.0 ** -40 * v.abs().sum(0)[:, None]
        t = 2.0 ** -8 * o.abs() + (torch.exp(2 * e) * (1 + 2.0 ** -10) - 1) * 2 * mag + tail
        outs.append(o.reshape(c.Hq, c.d))
        tols.append(t.reshape(c.Hq, c.d))
    return torch.stack(outs), torch.stack(tols)


@pytest.mark.parametrize("ratio", [4, 8, 10, 12, 14, 16, 18])
@pytest.mark.parametrize("Hq,Hkv,d", [(16, 4, 512), (24, 4, 512), (16, 8, 256), (32, 4, 256)])
@pytest.mark.parametrize("kvs", [False, True])
def test_a_channel_far_above_the_others(ratio, Hq, Hkv, d, kvs):
    c = Case(Hq, Hkv, d, [700, 40], kvs=kvs, seed=ratio, q_std=4.0, spread=0.2)
    c.q[..., 100] = 4.0 * 2.0 ** ratio * torch.where(c.q[..., 100] < 0, -1.0, 1.0).to(c.q.dtype)
    c.ks[..., 100 // 16] = 0
    got = c.run()[:, 0].double()
    want, tol = exact(c)
    over = (got - want).abs() - tol
    assert float(over.max()) <= 0, f"off by {float(over.max()):.3g} past the tolerance"


@pytest.mark.parametrize("Hq,Hkv,d", [(16, 4, 512), (32, 4, 256)])
def test_channels_spread_over_16_octaves(Hq, Hkv, d):
    """Every 16 dims at a size of their own, K the other way round, so that all count alike."""
    c = Case(Hq, Hkv, d, [700, 40], seed=3, q_std=4.0, spread=0.2)
    blocks = d // 16
    octave = (torch.arange(blocks, device="cuda") * 7 % 17).float()
    up = torch.exp2(octave - 16).repeat_interleave(16)
    c.q.mul_(up.to(c.q.dtype))
    s = 2.0 ** (7 - octave) * (0.75 + 0.5 * torch.rand(c.ks.shape, device="cuda", generator=torch.Generator(device="cuda").manual_seed(1)))
    c.ks.copy_(s.to(torch.float8_e4m3fn).view(torch.uint8))
    c.scale = c.scale * 2.0 ** 9
    got = c.run()[:, 0].double()
    want, tol = exact(c)
    over = (got - want).abs() - tol
    assert float(over.max()) <= 0, f"off by {float(over.max()):.3g} past the tolerance"
