"""Shared-prefix decodes in a row over buffers that are written again in front of
each: the own part starts before the prefix pass has ended, and must see what
was written before that."""
import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b
from test_gpu_shared import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch,fp8", [(2, False), (15, False), (40, False), (15, True), (40, True)])
def test_calls_in_a_row_see_what_was_written_before_each(batch, fp8):
    steps, n = 60, 300
    c = Case(16, 4, 512, [n] * batch, [0, batch], [2000], fp8=fp8, seed=batch, garbage=False)
    step = c.step()
    g = torch.Generator(device="cuda").manual_seed(3)
    qs = torch.randn((steps,) + tuple(c.q.shape), generator=g, device="cuda").to(torch.bfloat16)
    lens = torch.randint(1, n + 1, (steps, batch), generator=g, device="cuda", dtype=torch.int32)
    # the requests' tables change hands, and each one's newest row is written by the cache write
    tables = torch.stack([c.dev["table"][torch.randperm(batch, generator=g, device="cuda")] for _ in range(steps)])
    rows = torch.randn(steps, 2, batch, 4, 512, generator=g, device="cuda").to(torch.bfloat16)
    at = lens.long() - 1
    slots = (tables.gather(2, (at // 16)[:, :, None])[:, :, 0] * 16 + at % 16).to(torch.int32)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    pools = [c.kp.clone(), c.vp.clone()]
    desc = step.desc

    def run(apart):
        c.kp.copy_(pools[0])
        c.vp.copy_(pools[1])
        outs = [torch.empty_like(c.q) for _ in range(steps)]
        torch.cuda.synchronize()
        for i in range(steps):
            c.dev["table"].copy_(tables[i])
            c.dev["lens"].copy_(lens[i])
            c.q.copy_(qs[i])
            k, v = rows[i]
            if fp8:
                b.paged_decode_write_slots_fp8(desc, k, v, slots[i], c.kp, c.vp, c.ks, c.vs, flags)
            else:
                b.paged_decode_write_slots(desc, k, v, slots[i], c.kp, c.vp, flags)
            if apart:
                torch.cuda.synchronize()
            c.run(step, outs[i])
            if apart:
                torch.cuda.synchronize()
        assert step.check() == 0 and int(flags) == 0
        return outs

    alone = run(True)
    for _ in range(3):
        assert all(torch.equal(x.view(torch.int16), y.view(torch.int16)) for x, y in zip(run(False), alone))
