"""e4m3 shared-prefix decode whose answer hangs on pages with small V scales,
beside pages of the same prefix with large ones.

Tolerance, counted from the roundings (no own tokens, so the prefix pass's
alone): a token's operand is its probability times its V scale, relative to the
largest such product of its row in the piece or more, rounded to f16: 2^-12 of
itself, or half of f16's smallest step, 2^-25 of that product, for each of its
V codes; the other terms as in test_gpu_shared.py, with the output's 2^-8. So
    2^-8 |out| + (2^-12 + 2 ds + 2^-12) A + 2^-25 max_i (p_i s_i) sum_i |code_i|.
"""
import math

import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b
from test_gpu_shared import Case

pytestmark = pytest.mark.gpu


def _expect(c):
    """(out, tolerance) of requests without own tokens, one group."""
    B, Hkv, G = len(c.lens), c.Hkv, c.Hq // c.Hkv
    n = c.prefix[0]
    k = c._rows(c.kp, c.ks, c.ptab[0], n)
    codes, scale = (c.kp, c.ks) if c.kvs else (c.vp, c.vs)
    code = c._rows(codes, torch.ones_like(scale), c.ptab[0], n)
    page = torch.tensor(c.ptab[0], device="cuda")
    s_v = scale[page].double().repeat_interleave(c.P, 0)[:n]  # [n, Hkv]
    q = c.q.view(B, Hkv, G, c.d).double()
    s = torch.einsum("bhgd,nhd->bhgn", q, k) * c.scale
    a = torch.einsum("bhgd,nhd->bhgn", q.abs(), k.abs()) * abs(c.scale)
    w = torch.softmax(s, -1) * s_v.t()[None, :, None]
    e = torch.einsum("bhgn,nhd->bhgd", w, code)
    A = torch.einsum("bhgn,nhd->bhgd", w, code.abs())
    ds = (a.amax(-1) * c.d + 4 * (s.abs().amax(-1) + 8)) * 2.0 ** -24
    low = 2.0 ** -25 * w.amax(-1)[..., None] * code.abs().sum(0)[None, :, None]
    tol = 2.0 ** -8 * e.abs() + (2 * 2.0 ** -12 + 2 * ds[..., None]) * A + low
    return e.reshape(c.q.shape), tol.reshape(c.q.shape)


def _check(c, step=None):
    out, step = c.run(step)
    assert step.check() == 0
    e, tol = _expect(c)
    assert torch.isfinite(out).all()
    over = ((out.double() - e).abs() / tol.clamp(min=1e-300)).max().item()
    assert over <= 1.0, f"{over:.3f} of the tolerance"


def _peaked(Hq, Hkv, d, batch, kvs, at, jump, ratio, prefix=1200):
    """Every row's scores rise by `jump` nats at the page of token `at`, whose V scale is `ratio` of the others'."""
    c = Case(Hq, Hkv, d, [0] * batch, [0, batch], [prefix], fp8=True, kvs=kvs, seed=9, garbage=False)
    G, page = Hq // Hkv, c.ptab[0][at // 16]
    q = c.q.view(batch, Hkv, G, d)
    c.q.copy_(q[:1, :, :1].expand_as(q).reshape(c.q.shape))  # one direction per KV head
    u = c.q.view(batch, Hkv, G, d)[0, :, 0].float()
    rows = u / (u * u).sum(1, keepdim=True) * (jump * math.sqrt(d))
    if kvs:  # K = V: the page's scale is K's too, so the peak comes from the others' keys turning away
        c.ks *= 0.02 / c.ks.mean()
        flat = c.kp.view(torch.float8_e4m3fn).float()
        away = (-rows / 0.02).clamp(-448, 448)
        for p in c.ptab[0]:
            if p != page:
                flat[p] = away[:, None] * (1 + 0.1 * torch.randn(Hkv, 16, 1, device="cuda",
                                                                generator=torch.Generator("cuda").manual_seed(p)))
                c.ks[p] = 0.02
        c.kp.copy_(flat.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8))
        c.ks[page] = 0.02 * ratio
    else:
        big = rows.abs().amax(1)
        c.ks[page] = big / 448
        x = (rows / c.ks[page][:, None])[:, None].expand(-1, 16, -1)
        c.kp[page] = x.to(torch.float8_e4m3fn).view(torch.uint8)
        c.vs.copy_(torch.rand(c.vs.shape, device="cuda", generator=torch.Generator("cuda").manual_seed(3)) + 0.5)
        c.vs[page] = ratio
    return c


@pytest.mark.parametrize("batch", [3, 12, 40])
@pytest.mark.parametrize("at", [5, 900])
@pytest.mark.parametrize("jump,ratio", [(40.0, 1e-6), (40.0, 1e-8), (15.0, 1e-6), (12.0, 1e-4), (60.0, 2.0 ** -30)])
def test_peak_on_a_page_of_a_small_scale(batch, at, jump, ratio):
    _check(_peaked(16, 4, 512, batch, False, at, jump, ratio))


@pytest.mark.parametrize("at", [5, 900])
@pytest.mark.parametrize("ratio", [1e-5, 1e-8])
def test_peak_on_a_page_of_a_small_scale_key_is_value(at, ratio):
    _check(_peaked(16, 4, 512, 12, True, at, 40.0, ratio))


@pytest.mark.parametrize("Hq,Hkv,d", [(16, 8, 256), (32, 4, 256), (8, 2, 512)])
def test_other_layers(Hq, Hkv, d):
    _check(_peaked(Hq, Hkv, d, 5, False, 900, 40.0, 1e-7))


@pytest.mark.parametrize("batch", [3, 40])
def test_scales_that_fall_along_the_prefix(batch):
    """Page scales over nine orders of magnitude, scores that grow as the scales fall: each tile's products of
    probability and scale are about as large as the ones before."""
    c = Case(16, 4, 512, [0] * batch, [0, batch], [1600], fp8=True, seed=5, garbage=False)
    pages = torch.tensor(c.ptab[0], device="cuda")
    fall = torch.arange(100, device="cuda") / 99
    c.vs[pages] = (10.0 ** (-9 * fall))[:, None].expand(-1, 4)
    q = c.q.view(batch, 4, 4, 512)
    c.q.copy_(q[:1, :, :1].expand_as(q).reshape(c.q.shape))
    u = c.q.view(batch, 4, 4, 512)[0, :, 0].float()
    k = u / (u * u).sum(1, keepdim=True) * math.sqrt(512)
    x = k[None] * (9 * math.log(10.0) * fall)[:, None, None] + 1e-6
    c.ks[pages] = x.abs().amax(2) / 448
    c.kp[pages] = (x / c.ks[pages][:, :, None])[:, :, None].expand(-1, -1, 16, -1).to(torch.float8_e4m3fn).view(
        torch.uint8)
    _check(c)


@pytest.mark.parametrize("scale", [2.0 ** -120, 2.0 ** -130, 0.0])
def test_scales_near_the_end_of_fp32(scale):
    """Subnormal V scales give small finite rows. Flat scores: the rows' common factor, scale over 1200, then keeps
    2^-10 in fp32's subnormal numbers; the output's step there is 2^-133."""
    c = Case(16, 4, 512, [0] * 5, [0, 5], [1200], fp8=True, seed=5, q_std=0.0, garbage=False)
    c.vs.fill_(scale)
    out, step = c.run()
    assert step.check() == 0
    e, tol = _expect(c)
    assert ((out.double() - e).abs() <= tol + 2.0 ** -10 * e.abs() + 2.0 ** -134).all()


def test_the_longest_prefix():
    """2^31 - 256 tokens (every page the same few): the last steps of its loops pass 31 bits. Flat scores over one V
    code: the code's value. A piece's sums, below 2^24 and multiples of 24 below 2^25, are exact in fp32."""
    P, pages = 256, 2 ** 23 - 1
    kp = torch.zeros(4, 1, P, 256, dtype=torch.uint8, device="cuda")
    vp = torch.full_like(kp, 0x3c)  # 1.5
    scale = torch.ones(4, 1, device="cuda")
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    q = torch.ones(1, 1, 256, dtype=torch.bfloat16, device="cuda")
    step = b.SharedPrefixStep(1, 1, 256, P, 4, 1, [0], group_starts=[0, 1], prefix_lens=[pages * P],
                              max_prefix_pages=pages, kv_dtype=b.PD_KV_FP8_E4M3)
    tables = (torch.arange(pages, device="cuda") % 4).to(torch.int32).view(1, pages)
    out = step(q, kp, vp, tables, i32(pages * P), i32(0, 1), i32(-1).view(1, 1), i32(0), 1.0, torch.empty_like(q),
               k_scale=scale, v_scale=scale)
    assert step.check() == 0
    assert (out == 1.5).all()
