"""The slot, cache-write and shared-prefix calls launch on the current device:
tensors of another one are refused before the library is called (no GPU: stand-ins
for tensors, the current device and the library)."""

import struct

import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b


class OnGpu:
    """What the binding asks of a tensor, of one on GPU `device`."""

    def __init__(self, *shape, dtype=torch.int32, device=1, contiguous=True, token_stride=None):
        self.shape, self.dtype, self._device, self._contiguous = torch.Size(shape), dtype, device, contiguous
        self.device, self._token_stride = torch.device("cuda", device), token_stride
        n = 1
        for x in shape:
            n *= x
        self.nbytes = n * torch.empty(0, dtype=dtype).element_size()

    def get_device(self):
        return self._device

    def is_contiguous(self):
        return self._contiguous

    def data_ptr(self):
        return 1 << 20

    def dim(self):
        return len(self.shape)

    def stride(self):
        out, n = [], 1
        for x in reversed(self.shape):
            out.append(n)
            n *= x
        if self._token_stride is not None:
            out[-1] = self._token_stride
        return tuple(reversed(out))

    def numel(self):
        return self.nbytes // torch.empty(0, dtype=self.dtype).element_size()


class Library:
    """Counts the calls that reach it."""

    def __init__(self):
        self.calls = []

    def __getattr__(self, name):
        return lambda *a: self.calls.append((name,) + a) or b.PD_OK


BF16, U8 = torch.bfloat16, torch.uint8


def _append(at, stream, flags=None, workspace=None):
    i = lambda *s: OnGpu(*s, device=at)  # noqa: E731
    b.paged_decode_append_slots(16, 64, i(4), i(4), i(9), i(2), i(4, 8), i(4), i(5), i(32), i(32), i(2),
                                i(1) if flags is None else flags,
                                OnGpu(256, dtype=U8, device=at) if workspace is None else workspace, stream)


def _write(at, stream, flags=None):
    desc = b.layer_desc(16, 4, 512, 16, 4, 8)
    k, pool = OnGpu(3, 4, 512, dtype=BF16, device=at), OnGpu(4, 4, 16, 512, dtype=BF16, device=at)
    b.paged_decode_write_slots(desc, k, k, OnGpu(3, device=at), pool, pool,
                               OnGpu(1, device=at) if flags is None else flags, stream)


def _write_fp8(at, stream):
    desc = b.layer_desc(16, 4, 512, 16, 4, 8, 0, True, b.PD_KV_FP8_E4M3)
    pool, scale = OnGpu(4, 4, 16, 512, dtype=U8, device=at), OnGpu(4, 4, dtype=torch.float32, device=at)
    b.paged_decode_write_slots_fp8(desc, OnGpu(3, 4, 512, dtype=BF16, device=at), None, OnGpu(3, device=at), pool, None,
                                   scale, None, OnGpu(1, device=at), stream)


def _shared_plan(fp8=False):
    plan = b.SharedPlan()
    plan.own.layer = b.layer_desc(16, 4, 512, 16, 4, 8, 0, False, b.PD_KV_FP8_E4M3 if fp8 else b.PD_KV_BF16)
    plan.own.batch, plan.own.query_tokens, plan.num_groups, plan.max_prefix_pages = 2, 1, 1, 3
    return plan


def _shared_tensors(at, fp8=False):
    i = lambda *s: OnGpu(*s, device=at)  # noqa: E731
    pool = OnGpu(4, 4, 16, 512, dtype=U8 if fp8 else BF16, device=at)
    t = dict(q=OnGpu(2, 16, 512, dtype=BF16, device=at), k_pool=pool, v_pool=pool)
    if fp8:
        t["k_scale"] = t["v_scale"] = OnGpu(4, 4, dtype=torch.float32, device=at)
    return dict(t, prefix_tables=i(1, 3), prefix_lens=i(1), group_starts=i(2), block_tables=i(2, 8), seq_lens=i(2),
                workspace=OnGpu(4096, dtype=U8, device=at), out=OnGpu(2, 16, 512, dtype=BF16, device=at))


def _shared(at, stream):
    step, t = object.__new__(b.SharedPrefixStep), _shared_tensors(at)
    step.fp8, step.query_tokens, step.plan, step.workspace = False, 1, _shared_plan(), t.pop("workspace")
    step._shapes = b._SharedShapes(step.plan)
    step(scale=0.05, stream=stream, **t)


def _shared_call(at, stream, fp8=False, **kw):
    call = b.paged_decode_global_shared_fp8 if fp8 else b.paged_decode_global_shared
    call(_shared_plan(fp8), scale=0.05, stream=stream, **dict(_shared_tensors(at, fp8), **kw))


def _shared_call_fp8(at, stream):
    _shared_call(at, stream, True)


CALLS = [_append, _write, _write_fp8, _shared, _shared_call, _shared_call_fp8]


@pytest.fixture()
def library(monkeypatch):
    lib = Library()
    monkeypatch.setattr(b, "load_library", lambda *a: lib)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda device: 0, raising=False)
    return lib


@pytest.mark.parametrize("call", CALLS)
@pytest.mark.parametrize("stream", [None, 0, 1 << 12])
def test_tensors_of_another_device_than_the_current_one_are_refused(library, call, stream):
    with pytest.raises(ValueError, match="cuda:1"):
        call(1, stream)
    assert not library.calls
    call(0, stream)
    assert len(library.calls) == 1


@pytest.mark.parametrize("call", CALLS)
def test_a_stream_of_another_device_is_refused(library, call):
    class Stream:
        cuda_stream, device_index = 1 << 12, 1

    with pytest.raises(ValueError, match="cuda:1"):
        call(0, Stream())
    assert not library.calls
    Stream.device_index = 0
    call(0, Stream())
    assert len(library.calls) == 1


@pytest.mark.parametrize("call", [_append, _write])
@pytest.mark.parametrize("flags", [OnGpu(1, dtype=U8, device=0), OnGpu(0, device=0), OnGpu(3, dtype=U8, device=0),
                                   OnGpu(4, dtype=U8, device=0, contiguous=False), OnGpu(1, device=1)])
def test_flags_that_hold_no_word_are_refused(library, call, flags):
    with pytest.raises(ValueError, match="device_flags"):
        call(0, 0, flags=flags)
    assert not library.calls
    for good in (OnGpu(1, device=0), OnGpu(1, dtype=torch.uint32, device=0), OnGpu(16, dtype=U8, device=0)):
        call(0, 0, flags=good)
    assert len(library.calls) == 3


@pytest.mark.parametrize("workspace", [OnGpu(256, dtype=U8, device=0, contiguous=False), OnGpu(256, dtype=U8, device=1)])
def test_workspaces_that_are_not_one_piece_of_the_calls_gpu_are_refused(library, workspace):
    with pytest.raises(ValueError, match="workspace"):
        _append(0, 0, workspace=workspace)
    assert not library.calls


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("name,bad", [
    ("q", OnGpu(2, 16, 256, dtype=BF16, device=0)), ("q", OnGpu(2, 16, 512, dtype=torch.float16, device=0)),
    ("q", OnGpu(3, 16, 512, dtype=BF16, device=0)), ("out", OnGpu(1, 16, 512, dtype=BF16, device=0)),
    ("out", OnGpu(2, 16, 512, dtype=torch.float32, device=0)),
    ("out", OnGpu(2, 16, 512, dtype=BF16, device=0, contiguous=False)),
    ("k_pool", OnGpu(3, 4, 16, 512, dtype=BF16, device=0)), ("k_pool", OnGpu(3, 4, 16, 512, dtype=U8, device=0)),
    ("v_pool", OnGpu(4, 4, 16, 512, dtype=torch.float32, device=0)),
    ("prefix_tables", OnGpu(1, 2, device=0)), ("prefix_tables", OnGpu(1, 3, dtype=torch.int64, device=0)),
    ("prefix_lens", OnGpu(2, device=0)), ("group_starts", OnGpu(1, device=0)), ("block_tables", OnGpu(2, 4, device=0)),
    ("seq_lens", OnGpu(1, device=0)), ("seq_lens", OnGpu(2, device=1)), ("workspace", OnGpu(64, dtype=U8, device=0)),
    ("k_scale", OnGpu(4, 3, dtype=torch.float32, device=0)), ("v_scale", OnGpu(4, 4, dtype=BF16, device=0))])
def test_shared_calls_check_their_tensors(library, fp8, name, bad):
    if name.endswith("_scale") and not fp8:
        return
    with pytest.raises(ValueError, match=name):
        _shared_call(0, 0, fp8, **{name: bad}, workspace_bytes=4096)
    assert not library.calls
    _shared_call(0, 0, fp8, workspace_bytes=4096)
    assert len(library.calls) == 1


def test_shared_calls_take_addresses_and_leave_missing_tensors_to_the_library(library):
    t = {n: 1 << 20 for n in _shared_tensors(0) if n != "workspace"}
    _shared_call(0, 0, **t)
    _shared_call(0, 0, v_pool=None)
    assert len(library.calls) == 2
    t["q"] = None
    _shared_call(0, 0, **t)
    assert len(library.calls) == 3


def test_one_tokens_stride_may_be_anything(library):
    """A row of a tensor whose rows are no multiple of 8 elements apart is a whole row; two of them are not aligned."""
    desc, pool = b.layer_desc(16, 4, 512, 16, 4, 8), OnGpu(4, 4, 16, 512, dtype=BF16, device=0)
    strides = struct.Struct("P2i2P2q7P")

    def call(n, stride):
        k = OnGpu(n, 4, 512, dtype=BF16, device=0, token_stride=stride)
        b.paged_decode_write_slots(desc, k, k, OnGpu(n, device=0), pool, pool, OnGpu(1, device=0), 0)
        return strides.unpack(library.calls[-1][1])[5:7]

    for stride in (2052, 1, 0, 1 << 40):
        assert call(1, stride) == (2048, 2048)
    assert call(2, 2056) == (2056, 2056)
    assert call(2, 2052) == (2052, 2052)  # the library's to refuse
