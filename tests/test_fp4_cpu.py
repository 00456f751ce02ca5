"""The 4-bit cache's plans and refusals (no GPU): every bad argument is answered
before any CUDA call."""
import ctypes
import math
import shutil
import struct
import subprocess

import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b
from paged_gqa_decode_global_gb300 import build

FAKE = 1 << 20


@pytest.fixture(scope="module")
def lib():
    if torch.cuda.is_available():
        pytest.skip("a device is present: the accepted calls here have no memory behind their pointers")
    build.build()
    return b.load_library()


def _desc(**kw):
    a = dict(num_q_heads=16, num_kv_heads=4, head_dim=512, page_size=16, num_pages=64, max_pages_per_seq=8,
             kv_dtype=b.PD_KV_FP4_E2M1)
    a.update(kw)
    return b.layer_desc(**a)


# ---- plans


@pytest.mark.parametrize("kw,T", [
    (dict(head_dim=128), 1),              # fewer dims than a tile's slab
    (dict(head_dim=64), 1),
    (dict(num_q_heads=68, num_kv_heads=4), 1),   # 17 query heads a KV head
    (dict(num_pages=1 << 30), 1),         # pool rows past 31 bits
])
def test_plan_unsupported(lib, kw, T):
    with pytest.raises(b.PagedDecodeError) as e:
        b.paged_decode_plan_multi(_desc(**kw), T, [100, 20], 152)
    assert e.value.status == b.PD_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw,T,lens", [
    (dict(kv_dtype=3), 1, [10, 10]),
    (dict(page_size=24), 1, [10, 10]),
    (dict(), 1, [129, 10]),               # past the block table
    (dict(), 1, [-1, 10]),
    (dict(), 5, [4, 10]),                 # fewer cached than new
    (dict(), 0, [10, 10]),
    (dict(), 257, [10, 10]),
])
def test_plan_invalid(lib, kw, T, lens):
    with pytest.raises(b.PagedDecodeError) as e:
        b.paged_decode_plan_multi(_desc(**kw), T, lens, 152)
    assert e.value.status == b.PD_ERR_INVALID_ARG


def test_more_tiles_than_are_counted_are_refused(lib):
    # 65535 requests of a cap of 4 M tokens: 2^15 tiles each for 4 KV heads
    d = _desc(max_pages_per_seq=1 << 18, num_pages=1 << 20)
    b.paged_decode_plan(d, [1], 152)
    with pytest.raises(b.PagedDecodeError) as e:
        b.paged_decode_plan(d, [1] * 65535, 152)
    assert e.value.status == b.PD_ERR_UNSUPPORTED


@pytest.mark.parametrize("T,group,cc", [(1, 1, 4), (1, 4, 4), (2, 2, 4), (1, 5, 8), (2, 4, 8), (1, 16, 8), (256, 16, 8)])
@pytest.mark.parametrize("kvs", [False, True])
@pytest.mark.parametrize("d", [256, 512])
def test_plan_of_one_wave(lib, T, group, cc, kvs, d):
    pl = b.paged_decode_plan_multi(_desc(num_q_heads=4 * group, head_dim=d, kv_shared=kvs, max_pages_per_seq=64), T,
                                   [1024, T, 300], 152)
    assert (pl.grid_x, pl.grid_y, pl.grid_z, pl.num_splits, pl.merge_mode, pl.partial) == (152, 1, 1, 1, 0, 0)
    assert pl.chunk_tokens == 128 and pl.block_tokens == 16 and pl.query_tokens == T and pl.max_seq_len == 1024
    # one counter a CTA, then two pieces' log-sum-exps and rows
    assert pl.lse_offset >= 256 + 152 * 4
    assert pl.opart_offset - pl.lse_offset >= 152 * 2 * cc * 4
    assert pl.workspace_bytes == pl.opart_offset + 152 * 2 * cc * d * 4


def test_other_paths_refuse_the_cache(lib):
    d = _desc()
    with pytest.raises(b.PagedDecodeError) as e:
        b.paged_decode_plan_partial(d, [100, 20], 152)
    assert e.value.status == b.PD_ERR_UNSUPPORTED
    with pytest.raises(b.PagedDecodeError) as e:
        b.paged_decode_plan_shared(d, 1, [100, 20], [0, 2], [64], 8, 152)
    assert e.value.status == b.PD_ERR_UNSUPPORTED
    # the bf16 and e4m3 writes and decodes take their own layers only
    pl = b.paged_decode_plan(d, [100, 20], 152)
    f = ctypes.c_float(0.05)
    args = (FAKE, FAKE, FAKE + 4096, FAKE, FAKE, f, FAKE, 1 << 30, FAKE, None)
    assert lib.paged_decode_global(ctypes.byref(pl), *args) == b.PD_ERR_INVALID_ARG
    assert lib.paged_decode_write_slots(ctypes.byref(d), 5, FAKE, FAKE, 2048, 2048, FAKE, FAKE, FAKE + 4096, FAKE,
                                        None) == b.PD_ERR_INVALID_ARG


# ---- decode


DECODE = dict(q=FAKE, k=FAKE, v=FAKE + 4096, ks=FAKE + 8192, vs=FAKE + 12288, k_exp=0, v_exp=-4, tables=FAKE, lens=FAKE,
              scale=0.05, ws=FAKE, ws_bytes=1 << 30, out=FAKE, stream=None)


@pytest.mark.parametrize("kw,status", [(dict([(n, None)]), b.PD_ERR_INVALID_ARG) for n in
                                       ("q", "k", "v", "ks", "vs", "tables", "lens", "ws", "out")] + [
    (dict(q=FAKE + 8), b.PD_ERR_INVALID_ARG),
    (dict(k=FAKE + 8), b.PD_ERR_INVALID_ARG),
    (dict(ks=FAKE + 8), b.PD_ERR_INVALID_ARG),
    (dict(vs=FAKE + 8), b.PD_ERR_INVALID_ARG),
    (dict(v=FAKE), b.PD_ERR_INVALID_ARG),               # K's pool
    (dict(vs=FAKE + 8192), b.PD_ERR_INVALID_ARG),       # K's scales
    (dict(out=FAKE + 2), b.PD_ERR_INVALID_ARG),
    (dict(tables=FAKE + 2), b.PD_ERR_INVALID_ARG),
    (dict(k_exp=65), b.PD_ERR_INVALID_ARG),
    (dict(v_exp=-65), b.PD_ERR_INVALID_ARG),
    (dict(scale=math.nan), b.PD_ERR_INVALID_ARG),
    (dict(scale=math.inf), b.PD_ERR_INVALID_ARG),
    (dict(scale=3e38, k_exp=1), b.PD_ERR_INVALID_ARG),  # their product is infinite
    (dict(ws=FAKE + 128), b.PD_ERR_INVALID_ARG),
    (dict(ws_bytes=4096), b.PD_ERR_WORKSPACE_TOO_SMALL),
    (dict(), b.PD_ERR_CUDA),                            # accepted: gets as far as CUDA, absent here
])
@pytest.mark.parametrize("window", [0, 33])
def test_decode_refusals(lib, kw, status, window):
    a = dict(DECODE, **kw)
    a["scale"] = ctypes.c_float(a["scale"])
    pl = b.paged_decode_plan(_desc(window=window), [100, 20], 152)
    v = list(a.values())
    if window:
        assert lib.paged_decode_window_fp4(ctypes.byref(pl), *v[:9], window, *v[9:]) == status
        assert lib.paged_decode_window_fp4(ctypes.byref(pl), *v[:9], window + 1, *v[9:]) == b.PD_ERR_INVALID_ARG
        assert lib.paged_decode_global_fp4(ctypes.byref(pl), *v) == b.PD_ERR_INVALID_ARG
    else:
        assert lib.paged_decode_global_fp4(ctypes.byref(pl), *v) == status
        assert lib.paged_decode_window_fp4(ctypes.byref(pl), *v[:9], 33, *v[9:]) == b.PD_ERR_INVALID_ARG
    assert lib.paged_decode_global_fp4(None, *v) == b.PD_ERR_INVALID_ARG


def test_decode_of_a_shared_pool(lib):
    pl = b.paged_decode_plan(_desc(kv_shared=True), [100, 20], 152)

    def call(**kw):
        a = dict(DECODE, v=None, vs=None, v_exp=0, scale=ctypes.c_float(0.05))
        a.update(kw)
        return lib.paged_decode_global_fp4(ctypes.byref(pl), *a.values())

    assert call() == b.PD_ERR_CUDA
    assert call(v=FAKE, vs=FAKE + 8192) == b.PD_ERR_CUDA
    for bad in (dict(v=FAKE + 4096), dict(vs=FAKE + 12288), dict(v_exp=-1)):
        assert call(**bad) == b.PD_ERR_INVALID_ARG


@pytest.mark.parametrize("edit", [dict(magic=0), dict(version=99), dict(grid_x=0), dict(grid_x=5000), dict(grid_y=2),
                                  dict(num_splits=2), dict(merge_mode=1), dict(variant=0), dict(variant=61),
                                  dict(variant=68), dict(query_tokens=0), dict(batch=1 << 20), dict(lse_offset=256),
                                  dict(opart_offset=0), dict(workspace_bytes=1024), dict(smem_bytes=1024),
                                  dict(threads_per_cta=32), dict(partial=1), dict(block_tokens=64)])
def test_decode_refuses_a_plan_that_no_longer_agrees(lib, edit):
    pl = b.paged_decode_plan(_desc(), [100, 20], 152)
    for name, value in edit.items():
        setattr(pl, name, value)
    a = dict(DECODE, scale=ctypes.c_float(0.05))
    assert lib.paged_decode_global_fp4(ctypes.byref(pl), *a.values()) == b.PD_ERR_INVALID_ARG


# ---- rows by slot


ROWS = dict(n=5, k_exp=0, v_exp=-4, fp8=0, k=FAKE, v=FAKE, ks=2048, vs=2048, slots=FAKE, kp=FAKE, vp=FAKE + 4096,
            ksc=FAKE + 8192, vsc=FAKE + 12288, flags=FAKE, stream=0)


def _rows_call(lib, what, desc, kw):
    a = dict(ROWS, **kw)
    packed = b._ROWS_ARGS(ctypes.addressof(desc), a["n"], a["k_exp"], a["v_exp"], a["fp8"], a["k"] or 0, a["v"] or 0,
                          a["ks"], a["vs"], a["slots"] or 0, a["kp"] or 0, a["vp"] or 0, a["ksc"] or 0, a["vsc"] or 0,
                          a["flags"] or 0, 0)
    return (lib.paged_decode_write_slots_fp4_args if what == "write" else lib.paged_decode_read_slots_args)(packed)


@pytest.mark.parametrize("desc,kw,status", [
    (dict(), dict(n=-1), b.PD_ERR_INVALID_ARG),
    (dict(), dict(n=0, k=None, slots=None), b.PD_OK),
    (dict(), dict(k=None), b.PD_ERR_INVALID_ARG),
    (dict(), dict(v=None), b.PD_ERR_INVALID_ARG),
    (dict(), dict(slots=None), b.PD_ERR_INVALID_ARG),
    (dict(), dict(kp=None), b.PD_ERR_INVALID_ARG),
    (dict(), dict(vp=None), b.PD_ERR_INVALID_ARG),
    (dict(), dict(ksc=None), b.PD_ERR_INVALID_ARG),
    (dict(), dict(vsc=None), b.PD_ERR_INVALID_ARG),
    (dict(), dict(flags=None), b.PD_ERR_INVALID_ARG),
    (dict(), dict(k=FAKE + 8), b.PD_ERR_INVALID_ARG),
    (dict(), dict(kp=FAKE + 8), b.PD_ERR_INVALID_ARG),
    (dict(), dict(ksc=FAKE + 8), b.PD_ERR_INVALID_ARG),
    (dict(), dict(slots=FAKE + 2), b.PD_ERR_INVALID_ARG),
    (dict(), dict(vp=FAKE), b.PD_ERR_INVALID_ARG),           # K's pool
    (dict(), dict(vsc=FAKE + 8192), b.PD_ERR_INVALID_ARG),   # K's scales
    (dict(), dict(ks=2040), b.PD_ERR_INVALID_ARG),           # rows would overlap
    (dict(), dict(vs=2052), b.PD_ERR_INVALID_ARG),           # rows would lose their alignment
    (dict(), dict(ks=1 << 40), b.PD_ERR_INVALID_ARG),
    (dict(), dict(k_exp=65), b.PD_ERR_INVALID_ARG),
    (dict(), dict(v_exp=-65), b.PD_ERR_INVALID_ARG),
    (dict(head_dim=128), dict(), b.PD_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 28), dict(), b.PD_ERR_UNSUPPORTED),  # slots past 31 bits
    (dict(kv_shared=True), dict(), b.PD_ERR_INVALID_ARG),     # another pool for V
    (dict(kv_shared=True), dict(v=None, vp=None, vsc=None), b.PD_ERR_INVALID_ARG),  # exponents that differ
    (dict(kv_shared=True), dict(v=None, vp=None, vsc=None, v_exp=0), b.PD_ERR_CUDA),
    (dict(), dict(), b.PD_ERR_CUDA),                          # accepted
])
@pytest.mark.parametrize("what", ["write", "read"])
def test_rows_refusals(lib, what, desc, kw, status):
    assert _rows_call(lib, what, _desc(**desc), kw) == status


def test_rows_of_other_caches(lib):
    # the write takes a 4-bit layer only; the read what the layer says, with the scales that it has
    for kv in (b.PD_KV_BF16, b.PD_KV_FP8_E4M3):
        assert _rows_call(lib, "write", _desc(kv_dtype=kv), {}) == b.PD_ERR_INVALID_ARG
        assert _rows_call(lib, "read", _desc(kv_dtype=kv, head_dim=128), dict(ks=512, vs=512)) == b.PD_ERR_CUDA
    assert _rows_call(lib, "read", _desc(kv_dtype=3), {}) == b.PD_ERR_INVALID_ARG
    assert _rows_call(lib, "read", _desc(kv_dtype=b.PD_KV_FP8_E4M3), dict(ksc=None)) == b.PD_ERR_INVALID_ARG
    assert lib.paged_decode_write_slots_fp4_args(None) == b.PD_ERR_INVALID_ARG
    assert lib.paged_decode_read_slots_args(None) == b.PD_ERR_INVALID_ARG


def test_rows_arguments_lie_where_the_header_has_them(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    names = ("layer num_tokens k_exp v_exp {} k_rows v_rows k_stride v_stride slot_map k_pool v_pool k_scale v_scale "
             "device_flags stream").split()
    names.remove("{}")  # (the padding in front of the pointers)
    kinds = "P iii PP qq PPPPP PP".replace(" ", "")
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "paged_decode.h"', "int main(void) {"]
    lines += [f'  printf("%zu ", offsetof(pd_slot_rows_args, {m}));' for m in names]
    lines += ['  printf("%zu", sizeof(pd_slot_rows_args));', "  return 0;", "}"]
    (tmp_path / "l.c").write_text("\n".join(lines))
    subprocess.run([cc, "-I", build.INCLUDE, str(tmp_path / "l.c"), "-o", str(tmp_path / "l")], check=True)
    got = [int(x) for x in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True,
                                          check=True).stdout.split()]
    fmt = "P3i" + "i" + "2P2q7P"
    at, where = 0, []
    for k in "Piiii" + "PPqqPPPPPPP":
        size = struct.calcsize(k)
        at = (at + size - 1) // size * size
        where.append(at)
        at += size
    del where[4]  # the padding
    assert len(kinds) == len(names)
    assert got == where + [at]
    assert at == struct.calcsize(fmt) == len(b._ROWS_ARGS(*[0] * 16))


# ---- the binding


@pytest.mark.parametrize("largest,want", [(0.0, 0), (-1.0, 0), (math.nan, 0), (2688.0, 0), (2688.1, 1), (1344.0, -1),
                                          (1.0, -11), (1e-30, -64), (1e30, 64), (5376.0, 1)])
def test_exponent(largest, want):
    assert b.fp4_exponent(largest) == want


def test_binding_checks_tensors(lib):
    d = _desc(num_pages=4)
    z = lambda *s, t=torch.uint8: torch.zeros(*s, dtype=t)  # noqa: E731
    k, slots, flags = z(3, 4, 512, t=torch.bfloat16), z(3, t=torch.int32), z(1, t=torch.int32)
    pool, sc = z(4, 4, 16, 256), z(4, 4, 16, 32)
    good = dict(k=k, v=k.clone(), slots=slots, kp=pool, vp=pool.clone(), ks=sc, vs=sc.clone())
    for bad in (dict(k=k[..., :256]), dict(k=k.float()), dict(slots=slots.long()), dict(kp=z(4, 4, 16, 512)),
                dict(ks=z(4, 4, 16, 16)), dict(vs=sc.float()), dict(v=None), dict(vp=None), dict(vs=None)):
        a = dict(good, **bad)
        with pytest.raises(ValueError):
            b.paged_decode_write_slots_fp4(d, a["k"], a["v"], a["slots"], a["kp"], a["vp"], a["ks"], a["vs"], flags, 0)
        with pytest.raises(ValueError):
            b.paged_decode_read_slots_fp4(d, a["slots"], a["kp"], a["vp"], a["ks"], a["vs"], a["k"], a["v"], flags, 0)
    for what, kv in ((b.paged_decode_write_slots_fp4, b.PD_KV_BF16), (b.paged_decode_write_slots_fp4, b.PD_KV_FP8_E4M3)):
        with pytest.raises(ValueError, match="kv_dtype"):
            what(_desc(num_pages=4, kv_dtype=kv), k, k, slots, pool, pool, sc, sc, flags, 0)
    with pytest.raises(ValueError, match="GPU"):
        b.paged_decode_write_slots_fp4(d, k, k, slots, pool, pool.clone(), sc, sc.clone(), flags, 0)
    with pytest.raises(ValueError, match="kv_dtype"):
        b.paged_decode_read_slots(d, slots, pool, pool, k, k, flags, 0)
