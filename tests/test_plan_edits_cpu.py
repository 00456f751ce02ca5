"""Plans whose layer was edited after planning: what the planner refuses, every
launch refuses too, before any CUDA call."""
import ctypes

import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b

# addresses that are never followed: without a GPU an accepted call ends with PD_ERR_CUDA
pytestmark = pytest.mark.skipif(torch.cuda.is_available(), reason="made-up addresses")
FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    from paged_gqa_decode_global_gb300 import build
    build.build()
    return b.load_library()


def _plan(kv_dtype, T=1):
    d = b.layer_desc(16, 4, 512, 16, 64, 8, kv_dtype=kv_dtype)
    return b.paged_decode_plan_multi(d, T, [100, 20], 152)


def _call(lib, plan, kv_dtype):
    f = ctypes.c_float(0.05)
    tail = (FAKE, FAKE, f, FAKE, 1 << 40, FAKE, None)
    p = ctypes.byref(plan)
    if kv_dtype == b.PD_KV_BF16:
        return lib.paged_decode_global(p, FAKE, FAKE, FAKE + 4096, *tail)
    scaled = (FAKE, FAKE, FAKE + 4096, FAKE + 8192, FAKE + 12288)
    if kv_dtype == b.PD_KV_FP8_E4M3:
        return lib.paged_decode_global_fp8(p, *scaled, *tail)
    return lib.paged_decode_global_fp4(p, *scaled, 0, 0, *tail)


EDITS = [dict(page_size=24), dict(page_size=8), dict(page_size=0), dict(page_size=-16), dict(num_pages=0), dict(num_pages=-4),
         dict(max_pages_per_seq=0), dict(max_pages_per_seq=1 << 27),  # 2^31 tokens a request
         dict(max_pages_per_seq=1 << 28), dict(num_pages=1 << 26),    # 2^32 pool rows
         dict(num_pages=1 << 25, page_size=16), dict(num_pages=0x7fffffff, page_size=0x7ffffff0),
         dict(num_q_heads=0), dict(num_q_heads=-16), dict(num_kv_heads=0), dict(num_kv_heads=-4), dict(window=-1),
         dict(num_q_heads=65536, num_kv_heads=65536)]


@pytest.mark.parametrize("edit", EDITS)
@pytest.mark.parametrize("T", [1, 3])
@pytest.mark.parametrize("kv", [b.PD_KV_BF16, b.PD_KV_FP8_E4M3, b.PD_KV_FP4_E2M1])
def test_layer_edits_are_refused(lib, kv, T, edit):
    plan = _plan(kv, T)
    assert _call(lib, plan, kv) == b.PD_ERR_CUDA  # accepted: gets as far as CUDA, absent here
    for name, value in edit.items():
        setattr(plan.layer, name, value)
    assert _call(lib, plan, kv) == b.PD_ERR_INVALID_ARG


@pytest.mark.parametrize("kv", [b.PD_KV_BF16, b.PD_KV_FP8_E4M3, b.PD_KV_FP4_E2M1])
def test_the_largest_layers_are_not(lib, kv):
    plan = _plan(kv)
    plan.layer.num_pages = (1 << 25) - 1       # 2^31 - 64 pool rows
    plan.layer.max_pages_per_seq = (1 << 27) - 1
    assert _call(lib, plan, kv) == b.PD_ERR_CUDA
