"""Refusals of the slot-map, slot-write and shared-prefix calls (no GPU): every
bad argument is answered before any CUDA call, and the shared plan's fields."""
import ctypes

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


SLOT_ARGS = dict(batch=4, page_size=16, num_pages=64, max_pages=8, max_tokens=32, cached=FAKE, new=FAKE, free=FAKE,
                 num_free=10, rng=FAKE, tables=FAKE, lens=FAKE, starts=FAKE, slots=FAKE, pos=None, rng_out=FAKE,
                 flags=FAKE, ws=FAKE, ws_bytes=1 << 16, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), b.PD_ERR_INVALID_ARG),
    (dict(page_size=0), b.PD_ERR_INVALID_ARG),
    (dict(num_pages=0), b.PD_ERR_INVALID_ARG),
    (dict(max_pages=0), b.PD_ERR_INVALID_ARG),
    (dict(max_tokens=-1), b.PD_ERR_INVALID_ARG),
    (dict(num_free=-1), b.PD_ERR_INVALID_ARG),
    (dict(num_pages=1 << 30), b.PD_ERR_INVALID_ARG),   # slots past 31 bits
    (dict(max_pages=1 << 28), b.PD_ERR_INVALID_ARG),   # positions past 31 bits
    (dict(cached=None), b.PD_ERR_INVALID_ARG),
    (dict(new=None), b.PD_ERR_INVALID_ARG),
    (dict(free=None), b.PD_ERR_INVALID_ARG),
    (dict(rng=None), b.PD_ERR_INVALID_ARG),
    (dict(tables=None), b.PD_ERR_INVALID_ARG),
    (dict(lens=None), b.PD_ERR_INVALID_ARG),
    (dict(starts=None), b.PD_ERR_INVALID_ARG),
    (dict(slots=None), b.PD_ERR_INVALID_ARG),
    (dict(rng_out=None), b.PD_ERR_INVALID_ARG),
    (dict(flags=None), b.PD_ERR_INVALID_ARG),
    (dict(ws=None), b.PD_ERR_INVALID_ARG),
    (dict(ws=FAKE + 64), b.PD_ERR_INVALID_ARG),
    (dict(pos=FAKE + 2), b.PD_ERR_INVALID_ARG),
    (dict(cached=FAKE + 1), b.PD_ERR_INVALID_ARG),
    (dict(ws_bytes=16), b.PD_ERR_WORKSPACE_TOO_SMALL),
    (dict(), b.PD_ERR_CUDA),                           # accepted: gets as far as CUDA, absent here
])
def test_append_slots_refusals(lib, kw, status):
    a = dict(SLOT_ARGS, **kw)
    assert lib.paged_decode_append_slots(*a.values()) == status


def test_append_slots_workspace_grows_with_the_batch(lib):
    assert b.paged_decode_append_slots_workspace(0) >= 256
    assert b.paged_decode_append_slots_workspace(-5) >= 256
    assert b.paged_decode_append_slots_workspace(65535) % 256 == 0


def _desc(**kw):
    a = dict(num_q_heads=16, num_kv_heads=4, head_dim=512, page_size=16, num_pages=64, max_pages_per_seq=8)
    a.update(kw)
    return b.layer_desc(**a)


WRITE_ARGS = dict(n=5, k=FAKE, v=FAKE, ks=2048, vs=2048, slots=FAKE, kp=FAKE, vp=FAKE + 4096, flags=FAKE, stream=None)


@pytest.mark.parametrize("desc,kw,status", [
    (dict(), dict(n=-1), b.PD_ERR_INVALID_ARG),
    (dict(), dict(k=None), b.PD_ERR_INVALID_ARG),
    (dict(), dict(v=None), b.PD_ERR_INVALID_ARG),
    (dict(), dict(k=FAKE + 8), b.PD_ERR_INVALID_ARG),
    (dict(), dict(ks=2040), b.PD_ERR_INVALID_ARG),       # rows would overlap
    (dict(), dict(vs=2052), b.PD_ERR_INVALID_ARG),       # rows would lose their alignment
    (dict(), dict(ks=1 << 40), b.PD_ERR_INVALID_ARG),
    (dict(), dict(slots=None), b.PD_ERR_INVALID_ARG),
    (dict(), dict(kp=None), b.PD_ERR_INVALID_ARG),
    (dict(), dict(vp=None), b.PD_ERR_INVALID_ARG),
    (dict(), dict(vp=FAKE), b.PD_ERR_INVALID_ARG),       # V aliasing K on a K != V layer
    (dict(), dict(flags=None), b.PD_ERR_INVALID_ARG),
    (dict(kv_shared=True), dict(vp=FAKE + 4096), b.PD_ERR_INVALID_ARG),
    (dict(kv_dtype=b.PD_KV_FP8_E4M3), dict(), b.PD_ERR_INVALID_ARG),  # the bf16 call on an e4m3 layer
    (dict(head_dim=192), dict(), b.PD_ERR_UNSUPPORTED),
    (dict(num_pages=1 << 28), dict(), b.PD_ERR_UNSUPPORTED),
    (dict(page_size=0), dict(), b.PD_ERR_INVALID_ARG),
    (dict(), dict(n=0, k=None, slots=None), b.PD_OK),    # nothing to do
    (dict(kv_shared=True), dict(v=None, vp=None, vs=0), b.PD_ERR_CUDA),
    (dict(), dict(), b.PD_ERR_CUDA),
])
def test_write_slots_refusals(lib, desc, kw, status):
    a = dict(WRITE_ARGS, **kw)
    assert lib.paged_decode_write_slots(ctypes.byref(_desc(**desc)), *a.values()) == status


@pytest.mark.parametrize("kw,status", [
    (dict(sk=None), b.PD_ERR_INVALID_ARG),
    (dict(sv=None), b.PD_ERR_INVALID_ARG),
    (dict(sk=FAKE + 2), b.PD_ERR_INVALID_ARG),
    (dict(), b.PD_ERR_CUDA),
])
def test_write_slots_fp8_refusals(lib, kw, status):
    a = dict(n=5, k=FAKE, v=FAKE, ks=2048, vs=2048, slots=FAKE, kp=FAKE, vp=FAKE + 4096, sk=FAKE, sv=FAKE, flags=FAKE,
             stream=None)
    a.update(kw)
    d = _desc(kv_dtype=b.PD_KV_FP8_E4M3)
    assert lib.paged_decode_write_slots_fp8(ctypes.byref(d), *a.values()) == status
    assert lib.paged_decode_write_slots_fp8(ctypes.byref(_desc()), *a.values()) == b.PD_ERR_INVALID_ARG


def _plan(lens=(30, 40, 7), starts=(0, 2, 3), prefix=(160, 32), pages=10, T=1, sms=152, **kw):
    return b.paged_decode_plan_shared(_desc(**kw), T, list(lens), list(starts), list(prefix), pages, sms)


@pytest.mark.parametrize("kw,status", [
    (dict(starts=(1, 2, 3)), b.PD_ERR_INVALID_ARG),
    (dict(starts=(0, 2, 4)), b.PD_ERR_INVALID_ARG),
    (dict(starts=(0, 5, 3)), b.PD_ERR_INVALID_ARG),
    (dict(prefix=(161, 32)), b.PD_ERR_INVALID_ARG),     # not whole pages
    (dict(prefix=(176, 32)), b.PD_ERR_INVALID_ARG),     # past the table
    (dict(prefix=(-16, 32)), b.PD_ERR_INVALID_ARG),
    (dict(pages=0), b.PD_ERR_INVALID_ARG),
    (dict(lens=(30, 400, 7)), b.PD_ERR_INVALID_ARG),    # own tokens past their table
    (dict(T=8), b.PD_ERR_INVALID_ARG),                  # fewer own tokens than query tokens
    (dict(window=128), b.PD_ERR_UNSUPPORTED),
    (dict(head_dim=192), b.PD_ERR_UNSUPPORTED),
    (dict(num_q_heads=68), b.PD_ERR_UNSUPPORTED),
    (dict(head_dim=128, T=2), b.PD_ERR_UNSUPPORTED),
    (dict(sms=0), b.PD_ERR_INVALID_ARG),
])
def test_plan_shared_refusals(lib, kw, status):
    with pytest.raises(b.PagedDecodeError) as e:
        _plan(**kw)
    assert e.value.status == status


def test_plan_shared_covers_every_row_and_token(lib):
    for T, lens, starts, prefix in [(1, [9] * 40, [0, 40], [8000]), (3, [9] * 70, [0, 1, 33, 70], [16, 0, 4096]),
                                    (1, [1], [0, 0, 1], [32, 48]), (1, [0, 0], [0, 2], [0])]:
        pl = b.paged_decode_plan_shared(_desc(max_pages_per_seq=1000), T, lens, starts, prefix, 600, 152)
        per = T * 4
        rows = [(e - s) * per for s, e in zip(starts, starts[1:])]
        assert pl.tiles == sum(-(-r // pl.row_tile) for r in rows)
        longest = max([p for p, r in zip(prefix, rows) if r] + [0])
        assert pl.num_pieces * pl.chunk_tokens >= longest and pl.chunk_tokens % 128 == 0
        assert pl.own.partial == 2 and pl.own.merge_mode == 1
        n = len(lens) * T * 16
        assert pl.lse_offset >= pl.own.workspace_bytes and pl.o_offset >= pl.lse_offset + n * pl.num_pieces * 4
        assert pl.workspace_bytes >= pl.o_offset + n * pl.num_pieces * 512 * 4


SHARED_ARGS = dict(q=FAKE, k=FAKE, v=FAKE + 4096, ptab=FAKE, plens=FAKE, starts=FAKE, tables=FAKE, lens=FAKE,
                   scale=0.05, ws=FAKE, ws_bytes=1 << 30, out=FAKE, stream=None)


@pytest.mark.parametrize("kw,status", [(dict([(n, None)]), b.PD_ERR_INVALID_ARG) for n in
                                       ("q", "k", "v", "ptab", "plens", "starts", "tables", "lens", "ws", "out")] + [
    (dict(q=FAKE + 8), b.PD_ERR_INVALID_ARG),
    (dict(v=FAKE), b.PD_ERR_INVALID_ARG),
    (dict(starts=FAKE + 2), b.PD_ERR_INVALID_ARG),
    (dict(scale=float("nan")), b.PD_ERR_INVALID_ARG),
    (dict(scale=float("inf")), b.PD_ERR_INVALID_ARG),
    (dict(ws=FAKE + 16), b.PD_ERR_INVALID_ARG),
    (dict(ws_bytes=1024), b.PD_ERR_WORKSPACE_TOO_SMALL),
    (dict(), b.PD_ERR_CUDA),
])
def test_global_shared_refusals(lib, kw, status):
    a = dict(SHARED_ARGS, **kw)
    a["scale"] = ctypes.c_float(a["scale"])
    pl = _plan()
    assert lib.paged_decode_global_shared(ctypes.byref(pl), *a.values()) == status


def test_global_shared_refuses_a_plan_that_no_longer_agrees(lib):
    a = dict(SHARED_ARGS, scale=ctypes.c_float(0.05))

    def call(edit=None, **kw):
        pl = _plan(**kw)
        if edit:
            edit(pl)
        return lib.paged_decode_global_shared(ctypes.byref(pl), *a.values())

    def edit(path, value):
        def f(pl):
            obj = pl.own if path.startswith("own.") else pl
            setattr(obj, path.split(".")[-1], value)
        return f

    assert call(kv_dtype=b.PD_KV_FP8_E4M3) == b.PD_ERR_INVALID_ARG
    for path, value in (("num_pieces", 40), ("num_pieces", 0), ("chunk_tokens", 100), ("chunk_tokens", 0),
                        ("row_tile", 24), ("tiles", -1), ("tiles", 70000), ("magic", 0), ("version", 99),
                        ("workspace_bytes", 256), ("lse_offset", 0), ("num_groups", 0), ("own.partial", 1),
                        ("own.batch", 400), ("max_prefix_pages", 0)):
        assert call(edit(path, value)) == b.PD_ERR_INVALID_ARG, path
    # the own part is no plan for the calls that hand out partial results
    pl = _plan()
    assert lib.paged_decode_global_partial(ctypes.byref(pl.own), FAKE, FAKE, FAKE + 4096, FAKE, FAKE,
                                           ctypes.c_float(0.05), FAKE, 1 << 30, FAKE, FAKE,
                                           None) == b.PD_ERR_INVALID_ARG


def test_binding_checks_tensors(lib):
    d = _desc(num_pages=4)
    z = lambda *s, t=torch.bfloat16: torch.zeros(*s, dtype=t)  # noqa: E731
    k, pool, slots, flags = z(3, 4, 512), z(4, 4, 16, 512), z(3, t=torch.int32), z(1, t=torch.int32)
    for bad in (dict(k=z(3, 4, 256)), dict(k=z(3, 4, 512, t=torch.float32)), dict(k=z(3, 512, 4).transpose(1, 2)),
                dict(slots=z(3, t=torch.int64)), dict(pool=z(4, 4, 16, 256)), dict(v=None)):
        a = dict(k=k, v=k, slots=slots, pool=pool, vpool=pool.clone())
        a.update(bad)
        with pytest.raises(ValueError):
            b.paged_decode_write_slots(d, a["k"], a["v"], a["slots"], a["pool"], a["vpool"], flags, 0)
    i = lambda *s: z(*s, t=torch.int32)  # noqa: E731
    args = [i(4), i(4), i(9), i(2), i(4, 8), i(4), i(5), i(32), None, i(2), i(1), z(512, t=torch.uint8)]
    for at, bad in ((0, z(4, t=torch.int64)), (1, i(5)), (3, i(3)), (4, i(3, 8)), (6, i(4)), (8, i(31)), (9, i(1)),
                    (4, i(8, 4).t())):
        with pytest.raises(ValueError):
            b.paged_decode_append_slots(16, 64, *(args[:at] + [bad] + args[at + 1:]), stream=0)


def test_calls_by_structure(lib):
    # the structures are laid out as the binding packs them, and a missing one is refused
    calls = (lib.paged_decode_append_slots_args, lib.paged_decode_write_slots_args, lib.paged_decode_global_shared_args)
    packed = (b._SLOTS_ARGS(*[0] * 20), b._WRITE_ARGS(*[0] * 14), b._SHARED_ARGS(*[0] * 17))
    assert [len(x) for x in packed] == [136, 104, 128]
    for call, zeros in zip(calls, packed):
        assert call(None) != b.PD_OK
        assert call(zeros) != b.PD_OK  # page size 0, no layer, no plan


def test_tensors_on_the_host_are_refused(lib):
    i = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError, match="GPU"):
        b.paged_decode_append_slots(16, 64, i(4), i(4), i(9), i(2), i(4, 8), i(4), i(5), i(32), None, i(2), i(1),
                                    torch.zeros(512, dtype=torch.uint8), stream=0)
    k = torch.zeros(3, 4, 512, dtype=torch.bfloat16)
    pool = torch.zeros(4, 4, 16, 512, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="GPU"):
        b.paged_decode_write_slots(_desc(num_pages=4), k, k, i(3), pool, pool.clone(), i(1), 0)
