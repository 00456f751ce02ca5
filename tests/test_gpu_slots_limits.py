"""Slot maps at the ends of 31 bits."""
import pytest
import torch

from paged_gqa_decode_global_gb300 import binding as b

pytestmark = pytest.mark.gpu


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("P,cached", [(2 ** 31 - 1, 5), (2 ** 31 - 1, 2 ** 31 - 4), (2 ** 30 + 1, 2 ** 30 - 2)])
def test_pages_of_nearly_31_bits(P, cached):
    """The pages a request holds, where length + page size passes 31 bits: its tokens' page is its own first one."""
    table, lens, starts = _i32([[0]]), _i32([0]), _i32([0, 0])
    slots, pos, rng, flags = _i32([-7] * 4), _i32([-7] * 4), _i32([0, 0]), _i32([0])
    ws = torch.zeros(b.paged_decode_append_slots_workspace(1), dtype=torch.uint8, device="cuda")
    b.paged_decode_append_slots(P, 1, _i32([cached]), _i32([3]), _i32([0] * 8), _i32([0, 8]), table, lens, starts, slots,
                                pos, rng, flags, ws)
    want = [cached, cached + 1, cached + 2, -1]
    assert int(flags) == 0 and lens.tolist() == [cached + 3]
    assert slots.tolist() == want and pos.tolist() == want
    assert rng.tolist() == [0, 8] and table.tolist() == [[0]]


def test_a_request_without_new_pages_is_served_behind_the_end_of_the_longest_free_list():
    """One request finds no page left at entry 2^31 - 1; the next needs none, and
    its slot does not depend on how far the free list has been counted."""
    free = torch.empty(2 ** 31 - 1, dtype=torch.int32, device="cuda")
    table, lens, starts = _i32([[3, -1], [5, -1]]), _i32([0, 0]), _i32([0, 0, 0])
    slots, pos, rng, flags = _i32([-7] * 4), _i32([-7] * 4), _i32([0, 0]), _i32([0])
    ws = torch.zeros(b.paged_decode_append_slots_workspace(2), dtype=torch.uint8, device="cuda")
    b.paged_decode_append_slots(16, 8, _i32([16, 4]), _i32([1, 2]), free, _i32([2 ** 31 - 1, 2 ** 31 - 1]), table, lens,
                                starts, slots, pos, rng, flags, ws)
    assert int(flags) == b.PD_DEVFLAG_NO_PAGES
    assert lens.tolist() == [16, 6] and starts.tolist() == [0, 1, 3]
    assert slots.tolist() == [-1, 5 * 16 + 4, 5 * 16 + 5, -1] and pos.tolist() == [-1, 4, 5, -1]
    assert rng.tolist() == [2 ** 31 - 1] * 2 and table.tolist() == [[3, -1], [5, -1]]
