"""The e4m3 cache write code by code: every bf16 value under scales of every
size, against the quotient's own rounding. The quotient in 64 bits, rounded to
fp32, is the correctly rounded fp32 quotient (53 bits hold a 24-bit quotient's
rounding: 2 * 24 + 2), and the e4m3 code is looked up among all of them: no
tolerance. Values are shuffled, so that a thread's 16 elements hold ordinary
magnitudes and extremes side by side; infinities and NaN, which take the
division, are apart from them."""
import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b

pytestmark = pytest.mark.gpu

P, D = 16, 128
# around the reciprocal path's ends (2^-60, 2^60), ordinary ones, far ones, subnormal, zero, negative
SCALES = [2.0 ** -60, 2.0 ** -60 * (1 + 2.0 ** -23), 1e-17, 1e-9, 1.3e-5, 1e-3, 0.0071, 1 / 3, 0.5, 1.0, 1.7, 3.0, 448.0,
          1e9, 2.0 ** 60 * (1 - 2.0 ** -24), 2.0 ** 60, 1e-30, 1e30, 1e-40, 0.0, -0.0, -0.37, -2e-8, float("inf")]


def _codes(x, scale):
    """The e4m3 code of each fp32 quotient x / scale: nearest, ties to the even code, clamped, the sign the quotient's."""
    q = (x.double() / scale.double()).float()
    table = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    m = q.abs().double().clamp(max=448.0).nan_to_num(0.0)
    hi = torch.searchsorted(table, m).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    up, down = table[hi] - m, m - table[lo]
    code = torch.where((up < down) | ((up == down) & (hi % 2 == 0)), hi, lo)
    code = code | (torch.signbit(q).long() << 7)
    return torch.where(q.isnan(), torch.full_like(code, 0x7f), code).to(torch.uint8)


def _write(x, scales):
    """Codes of x [n, D] under each scale in turn: [scales, n, D]."""
    n, pages = x.shape[0], -(-x.shape[0] // P)
    pool = torch.zeros(len(scales) * pages, 1, P, D, dtype=torch.uint8, device="cuda")
    ks = torch.tensor(scales, dtype=torch.float32).repeat_interleave(pages).view(-1, 1).cuda()
    k = x.repeat(len(scales), 1).view(-1, 1, D).cuda()
    slots = (torch.arange(len(scales))[:, None] * pages * P + torch.arange(n)).view(-1).to(torch.int32).cuda()
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    b.paged_decode_write_slots_fp8(b.layer_desc(1, 1, D, P, pool.shape[0], 8, 0, True, b.PD_KV_FP8_E4M3), k, None,
                                   slots, pool, None, ks, None, flags)
    torch.cuda.synchronize()
    assert int(flags) == 0
    return pool.view(len(scales), pages * P, D)[:, :n].cpu()


def _finite():
    bits = torch.arange(1 << 16, dtype=torch.int32)
    bits = bits[(bits & 0x7f80) != 0x7f80]
    return bits[torch.randperm(bits.numel(), generator=torch.Generator().manual_seed(1))]


def _rows(bits):
    """The bf16 of these bit patterns in rows of D, filled up with ones."""
    bits = torch.cat([bits, torch.full((-bits.numel() % D,), 0x3f80, dtype=torch.int32)])
    return torch.where(bits >= 1 << 15, bits - (1 << 16), bits).to(torch.int16).view(torch.bfloat16).view(-1, D)


def _differ(got, x, nonzero):
    """(scale, value, code, expected) where they differ, at values whose quotients are (not) zero."""
    bad = []
    for i, s in enumerate(SCALES):
        e = _codes(x.float(), torch.tensor(s, dtype=torch.float32))
        g, nan = got[i], e == 0x7f
        same = torch.where(nan, (g & 0x7f) == 0x7f, g == e) | ((x == 0) & ~nan & bool(nonzero))
        if not nonzero:
            same |= x != 0
        bad += [(s, float(x[~same][j]), int(g[~same][j]), int(e[~same][j])) for j in range(min(3, int((~same).sum())))]
    return bad


def test_every_finite_value_has_its_quotients_code():
    """Values whose quotients pass the fp32 range clamp like any other, whatever stands beside them."""
    x = _rows(_finite())
    assert not _differ(_write(x, SCALES), x, True)


def test_infinities_and_nan_beside_ordinary_values():
    bits = _finite()[:2000]
    bits[::16] = torch.tensor([0x7f80, 0xff80, 0x7fc0, 0xffc1, 0x7f81], dtype=torch.int32).repeat(25)
    x = _rows(bits)
    assert not _differ(_write(x, SCALES), x, True)


def test_zeros_keep_their_quotients_sign():
    """A zero's code has the sign of its quotient, whichever way its neighbours send it."""
    bits = _finite()[:4000]
    bits[::3] = torch.tensor([0x0000, 0x8000], dtype=torch.int32)[torch.arange(1334) % 2]
    bits = torch.cat([bits, torch.tensor([0x0000, 0x8000] * 64, dtype=torch.int32)])
    ordinary = bits & 0x7fff
    bits[2000:4000] = torch.where(ordinary[2000:4000] >= 0x6000, 0x8000, bits[2000:4000])  # no value near the ends
    x = _rows(bits)
    assert not _differ(_write(x, SCALES), x, False)
