"""Where the plans of all caches lay out a workspace that they may take in turn: the
4-bit decode's counts, a byte a CTA behind the error word, have to stay out of
reach of the others' pieces."""
import pytest

from paged_gqa_decode_global_gb300 import binding as b

HEADER = 256


def _desc(kv_dtype, **kw):
    a = dict(num_q_heads=16, num_kv_heads=4, head_dim=512, page_size=16, num_pages=8192, max_pages_per_seq=2048,
             kv_dtype=kv_dtype)
    a.update(kw)
    return b.layer_desc(**a)


@pytest.fixture(scope="module", autouse=True)
def _built():
    from paged_gqa_decode_global_gb300 import build
    build.build()


@pytest.mark.parametrize("sms", [1, 2, 40, 152, 255, 256, 300, 4096, 5000, 1 << 20])
@pytest.mark.parametrize("T,d", [(1, 512), (2, 512), (64, 256)])
def test_counts_fit_the_header(sms, T, d):
    pl = b.paged_decode_plan_multi(_desc(b.PD_KV_FP4_E2M1, head_dim=d), T, [32768] * 4, sms)
    assert 1 <= pl.grid_x <= sms
    assert 4 + pl.grid_x <= HEADER <= pl.lse_offset
    assert pl.grid_x == sms or pl.grid_x >= 152  # every SM of a GB300 has a share


@pytest.mark.parametrize("sms", [1, 40, 152, 1000])
@pytest.mark.parametrize("kv", [b.PD_KV_BF16, b.PD_KV_FP8_E4M3])
def test_other_plans_begin_behind_it(sms, kv):
    plans = [b.paged_decode_plan(_desc(kv), lens, sms) for lens in ([9000], [2000] * 8, [32768] * 4, [300, 17])]
    plans.append(b.paged_decode_plan_multi(_desc(kv), 3, [9000], sms))
    shared = b.paged_decode_plan_shared(_desc(kv), 1, [100] * 16, [0, 16], [4096], 256, sms)
    plans.append(shared.own)
    if kv == b.PD_KV_BF16:
        plans.append(b.paged_decode_plan_partial(_desc(kv), [9000], sms))
    for pl in plans:
        assert pl.lse_offset >= HEADER and pl.opart_offset >= HEADER and pl.workspace_bytes >= HEADER
    assert shared.lse_offset >= HEADER and shared.o_offset >= HEADER
