"""Shared-prefix plans edited by hand (no GPU)."""
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


def test_a_plan_without_row_tiles_is_refused(lib):
    """Without a prefix pass in front of it the own part would wait for nothing."""
    desc = b.layer_desc(16, 4, 512, 16, 64, 8)

    def call(tiles=None, lens=(30, 40, 7), starts=(0, 2, 3)):
        plan = b.paged_decode_plan_shared(desc, 1, list(lens), list(starts), [160, 32], 10, 152)
        plan.tiles = plan.tiles if tiles is None else tiles
        return lib.paged_decode_global_shared(ctypes.byref(plan), FAKE, FAKE, FAKE + 4096, FAKE, FAKE, FAKE, FAKE, FAKE,
                                              ctypes.c_float(0.05), FAKE, 1 << 30, FAKE, None)

    assert call() == b.PD_ERR_CUDA  # accepted: gets as far as CUDA, absent here
    assert call(tiles=0) == b.PD_ERR_INVALID_ARG
    assert call(lens=(), starts=(0, 0, 0)) == b.PD_OK  # no requests, no tiles
