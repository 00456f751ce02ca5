"""A NaN score stays its rows' result however little its piece of the prefix weighs."""
import pytest
import torch

from test_gpu_shared import Case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("batch", [3, 15, 40])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("token", [3, 40])
def test_a_nan_key_is_not_lost_behind_a_peak(batch, fp8, token):
    """Behind the NaN, scores rise by 200 nats: in its own piece (its row's sum is begun anew there), and by 300 more in
    another, next to which the piece weighs nothing."""
    c = Case(16, 4, 512, [7] * batch, [0, batch], [8000], fp8=fp8, seed=9, garbage=False)
    step = c.step()
    assert step.plan.num_pieces > 1 and step.plan.chunk_tokens >= 256
    q = c.q.view(batch, 4, 4, 512)
    c.q.copy_(q[:1, :, :1].expand_as(q).reshape(c.q.shape))  # one direction per KV head
    u = c.q.view(batch, 4, 4, 512)[0, :, 0].float()
    unit = u / (u * u).sum(1, keepdim=True) * 512 ** 0.5
    # every token of the pages has the page's score, so that each lane has one
    for page, score in ((c.ptab[0][i], 200.0) for i in range(8, 16)):
        _set(c, page, unit * score)
    _set(c, c.ptab[0][-1], unit * 500.0)
    finite, _ = c.run(step)
    assert torch.isfinite(finite).all()
    c.kp[c.ptab[0][token // 16], 2, token % 16] = 0x7f if fp8 else float("nan")
    out, _ = c.run(step)
    assert step.check() == 0
    assert out[:, 8:12].isnan().all()
    keep = [h for h in range(16) if not 8 <= h < 12]
    assert torch.equal(out[:, keep], finite[:, keep])


def _set(c, page, rows):
    """Every token of a page gets this key per KV head."""
    if c.fp8:
        c.ks[page] = rows.abs().amax(1) / 448
        x = (rows / c.ks[page][:, None])[:, None].expand(-1, 16, -1)
        c.kp[page] = x.to(torch.float8_e4m3fn).view(torch.uint8)
    else:
        c.kp[page] = rows[:, None].expand(-1, 16, -1).to(torch.bfloat16)
