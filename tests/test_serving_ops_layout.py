"""The binding's packed arguments and structures against the header as a C
compiler lays it out (no GPU)."""
import ctypes
import shutil
import struct
import subprocess

import pytest

from paged_gqa_decode_global_gb300 import binding as b
from paged_gqa_decode_global_gb300 import build

# what the binding packs, in its order (binding.py: the calls of _SLOTS_ARGS, _WRITE_ARGS and _SHARED_ARGS)
PACKED = {
    "pd_append_slots_args": ("6i12PQP", b._SLOTS_ARGS, "batch page_size num_pages max_pages max_tokens num_free "
                             "cached_lens new_tokens free_pages free_range block_tables seq_lens token_starts slot_map "
                             "positions free_range_out device_flags workspace workspace_bytes stream"),
    "pd_write_slots_args": ("P2i2P2q7P", b._WRITE_ARGS, "layer num_tokens fp8 k_in v_in k_stride v_stride slot_map "
                            "k_pool v_pool k_scale v_scale device_flags stream"),
    "pd_global_shared_args": ("P10PfiPQ2P", b._SHARED_ARGS, "plan q k_pool v_pool k_scale v_scale prefix_tables "
                              "prefix_lens group_starts block_tables seq_lens scale fp8 workspace workspace_bytes out "
                              "stream"),
}
STRUCTURES = {"pd_layer_desc": b.LayerDesc, "pd_plan": b.Plan, "pd_shared_plan": b.SharedPlan}


def _fields(fmt):
    """The size of each value of a native-alignment struct format, one by one, and where it lies."""
    kinds, count = [], ""
    for ch in fmt:
        if ch.isdigit():
            count += ch
        else:
            kinds += [ch] * int(count or 1)
            count = ""
    return [(struct.calcsize("".join(kinds[:i + 1])) - struct.calcsize(k), struct.calcsize(k))
            for i, k in enumerate(kinds)], struct.calcsize(fmt)


@pytest.fixture(scope="module")
def header(tmp_path_factory):
    """{structure: (size, {member: (offset, size)})} as the C compiler sees the header."""
    cc = shutil.which("gcc") or shutil.which("cc")
    if cc is None:
        pytest.skip("no C compiler")
    want = {n: names.split() for n, (_, _, names) in PACKED.items()}
    want.update({n: [f[0] for f in s._fields_] for n, s in STRUCTURES.items()})
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "paged_decode.h"', "int main(void) {"]
    for n, members in want.items():
        lines.append(f'  printf("{n} - %zu 0\\n", sizeof({n}));')
        lines += [f'  printf("{n} {m} %zu %zu\\n", offsetof({n}, {m}), sizeof((({n}*)0)->{m}));' for m in members]
    d = tmp_path_factory.mktemp("layout")
    (d / "layout.c").write_text("\n".join(lines + ["  return 0;", "}"]))
    subprocess.run([cc, "-I", build.INCLUDE, str(d / "layout.c"), "-o", str(d / "layout")], check=True)
    out = {}
    for line in subprocess.run([str(d / "layout")], check=True, capture_output=True, text=True).stdout.splitlines():
        n, m, at, size = line.split()
        if m == "-":
            out[n] = (int(at), {})
        else:
            out[n][1][m] = (int(at), int(size))
    return out


@pytest.mark.parametrize("name", PACKED)
def test_packed_arguments_lie_where_the_header_has_them(header, name):
    fmt, pack, names = PACKED[name]
    places, size = _fields(fmt)
    total, members = header[name]
    assert places == [members[m] for m in names.split()]
    assert size == total == len(pack(*[0] * len(places)))
    # the format is the packer's own: each value at its place
    raw = pack(*range(1, len(places) + 1))
    assert list(struct.unpack(fmt, raw)) == list(range(1, len(places) + 1))


@pytest.mark.parametrize("name", STRUCTURES)
def test_structures_lie_where_the_header_has_them(header, name):
    cls = STRUCTURES[name]
    total, members = header[name]
    assert ctypes.sizeof(cls) == total
    for f, _ in cls._fields_:
        at = getattr(cls, f)
        assert (at.offset, at.size) == members[f], f


def test_append_slots_workspace_holds_its_counter():
    """One 32-bit counter whatever the batch, in a 256-byte aligned buffer."""
    build.build()
    assert {b.paged_decode_append_slots_workspace(n) for n in (0, 1, 1024, 65535, 2 ** 31 - 1)} == {256}
