"""One workspace taken in turn by plans of every kind: the 4-bit decode's counts
survive the others' pieces. Each output has the bits that its plan gives on a
workspace of its own, where it is held against 64 bits by the tests of its kind."""
import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b
from paged_gqa_decode_global_gb300 import inputs as synth
from test_gpu_fp4 import Case, compare
from test_gpu_shared import Case as SharedCase

pytestmark = pytest.mark.gpu


def four_bits(sms, lens, **kw):
    c = Case(16, 4, 512, lens, seed=sms + len(lens), **kw)
    plan = c.step(sm_count=sms).plan

    def run(ws):
        q = c.q if c.T > 1 else c.q[:, 0]
        out = torch.full_like(q, 7.0)
        a = (plan, q, c.kc, c.vc, c.ks, c.vs, c.table, c.lens)
        if c.window:
            b.paged_decode_window_fp4(*a, c.window, c.scale, ws, out)
        else:
            b.paged_decode_global_fp4(*a, c.scale, ws, out)
        return out

    def right(out):
        compare(c, out.view(c.q.shape))

    return plan, run, right


def two_kernels(fp8):
    """A bf16 or e4m3 plan whose pieces the merge kernel joins (out of the workspace)."""
    lens = [9000]
    li = synth.make_layer("ws", lens, 16, 4, 512, pool_pages=600, seed=11, device="cuda")
    li = synth.quantize_kv_fp8(li) if fp8 else li
    step = b.LayerStep.for_inputs(li, sm_count=1000)
    assert step.plan.merge_mode == 1

    def run(ws):
        out = torch.full_like(li.q, 7.0)
        if fp8:
            b.paged_decode_global_fp8(step.plan, li.q, li.k8, li.v8, li.k_scale, li.v_scale, li.block_tables,
                                      li.seq_lens, li.scale, ws, out)
        else:
            b.paged_decode_global(step.plan, li.q, li.k_pool, li.v_pool, li.block_tables, li.seq_lens, li.scale, ws, out)
        b.paged_decode_merge(step.plan, ws, out)
        return out

    return step.plan, run, None


def shared_prefix(fp8):
    c = SharedCase(16, 4, 512, [300] * 16, [0, 16], [2000], seed=4, fp8=fp8)
    plan, v = c.step().plan, c.dev

    def run(ws):
        out = torch.full_like(c.q, 7.0)
        a = (v["ptab"], v["plens"], v["starts"], v["table"], v["lens"], c.scale, ws, out)
        if fp8:
            b.paged_decode_global_shared_fp8(plan, c.q, c.kp, c.vp, c.ks, c.vs, *a)
        else:
            b.paged_decode_global_shared(plan, c.q, c.kp, c.vp, *a)
        return out

    return plan, run, None


def kinds():
    return [four_bits(152, [3000, 500, 9000]), two_kernels(False), four_bits(40, [2500, 1900]), two_kernels(True),
            four_bits(152, [20000], kvs=True), shared_prefix(False), four_bits(300, [1111, 640, 128]), shared_prefix(True),
            four_bits(7, [2000, 33, 2000], T=3, window=1000), four_bits(1, [700])]


def test_plans_of_every_kind_take_one_workspace_in_turn():
    all_of_them = kinds()
    size = (max(int(p.workspace_bytes) for p, _, _ in all_of_them) + 255) // 256 * 256
    want = []
    for _, run, right in all_of_them:
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        want.append(run(ws))
        if right:
            right(want[-1])
    ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    for _ in range(3):
        for i, (plan, run, _) in enumerate(all_of_them):
            assert torch.equal(run(ws).view(torch.int16), want[i].view(torch.int16)), i
        assert int(ws[:256].count_nonzero()) == 0  # no error, no count left
    for (plan, run, _), w in reversed(list(zip(all_of_them, want))):
        assert torch.equal(run(ws).view(torch.int16), w.view(torch.int16))
        own = plan.own if isinstance(plan, b.SharedPlan) else plan
        assert b.paged_decode_check_device_error(own, ws) == 0


def test_two_graphs_of_two_kinds_share_a_workspace():
    pair = [four_bits(152, [3000, 500, 9000]), two_kernels(False)]
    size = max(int(p.workspace_bytes) for p, _, _ in pair)
    ws = torch.zeros((size + 255) // 256 * 256, dtype=torch.uint8, device="cuda")
    want = [run(torch.zeros_like(ws)) for _, run, _ in pair]
    graphs, outs = [], []
    for _, run, _ in pair:
        run(ws)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(run(ws))
        graphs.append(g)
    for _ in range(4):
        for g, out, w in zip(graphs, outs, want):
            out.fill_(9.0)
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out.view(torch.int16), w.view(torch.int16))


def test_another_plan_sets_the_counts_back_after_a_time_out():
    c = Case(16, 4, 512, [3000, 900], seed=5)
    step, (other, run, _) = c.step(), two_kernels(False)
    size = (max(int(other.workspace_bytes), int(step.plan.workspace_bytes)) + 255) // 256 * 256
    step.workspace = ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
    want = c.run(step).clone()
    step.plan.test_stall_bytes = 16
    c.run(step, check=False)
    step.plan.test_stall_bytes = 0
    run(ws)
    with pytest.raises(b.PagedDecodeError) as e:
        b.paged_decode_check_device_error(other, ws)
    assert e.value.flags & b.PD_DEVFLAG_WAIT_TIMEOUT
    assert int(ws[:256].count_nonzero()) == 0
    for _ in range(3):
        assert torch.equal(c.run(step), want)
