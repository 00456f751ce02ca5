"""The serving loop (slots, cache writes and shared-prefix decode together)
against attention over each request's rows in 64 bits, and the bounded waits of
the prefix pass.

Tolerance as in test_gpu_shared.py: e = 2^-8 of the output, e A for the
probabilities' rounding, 2^-9 A for scores, exponentials and sums at these
sizes (|score| < 2^4, d = 512: 2 ds < 2^-10; 2^-12 for sums)."""
import time

import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b
from paged_gqa_decode_global_gb300 import serving_step
from test_gpu_shared import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kw", [dict(), dict(batch=1, prompt_tokens=16, steps=3), dict(batch=40, prompt_tokens=1040),
                                dict(batch=3, prompt_tokens=0, tails=[15, 16, 17], steps=5)])
def test_serving_loop(kw):
    for s in serving_step.run(seed=3, **kw):
        q, out = s["q"].double(), s["out"].double()
        for r, (k, v) in enumerate(zip(s["k"], s["v"])):
            k, v = k.double(), v.double()
            qr = q[r].view(k.shape[1], -1, k.shape[2])
            w = torch.softmax(torch.einsum("hgd,nhd->hgn", qr, k) * k.shape[2] ** -0.5, -1)
            e = torch.einsum("hgn,nhd->hgd", w, v).reshape(out[r].shape)
            A = torch.einsum("hgn,nhd->hgd", w, v.abs()).reshape(out[r].shape)
            assert ((out[r] - e).abs() <= 2.0 ** -8 * e.abs() + (2.0 ** -8 + 2.0 ** -9) * A).all()


@pytest.mark.parametrize("rows,fp8", [(2, False), (20, False), (2, True), (20, True)])
def test_waits_run_out_and_report(rows, fp8):
    """Copies that never deliver all the bytes a stage expects: every wait of the
    prefix pass (one CTA, and a pair) and of the own part runs out, the error
    word says so, and the next call is right again."""
    c = Case(16, 4, 512, [20] * rows, [0, rows], [528], seed=2, fp8=fp8)
    step = c.step()
    step.plan.own.test_stall_bytes = 16
    began = time.monotonic()
    c.run(step)
    with pytest.raises(b.PagedDecodeError) as e:
        step.check()
    assert e.value.flags & b.PD_DEVFLAG_WAIT_TIMEOUT
    assert time.monotonic() - began < 30
    step.plan.own.test_stall_bytes = 0
    c.check(step)
