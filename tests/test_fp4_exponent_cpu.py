"""The exponent of a 4-bit layer at the ends of its range."""
import math

import pytest

from paged_gqa_decode_global_gb300 import binding as b


@pytest.mark.parametrize("largest,want", [(math.inf, 64), (-math.inf, 0), (2688.0 * 2.0 ** 64, 64), (2688.0 * 2.0 ** 65, 64),
                                          (1.7e308, 64), (2688.0 * 2.0 ** -64, -64), (5e-324, -64)])
def test_ends(largest, want):
    assert b.fp4_exponent(largest) == want


@pytest.mark.parametrize("e", range(-63, 64))
def test_every_exponent_is_the_smallest(e):
    assert b.fp4_exponent(math.ldexp(2688.0, e)) == e
    assert b.fp4_exponent(math.nextafter(math.ldexp(2688.0, e), math.inf)) == e + 1
    assert b.fp4_exponent(math.nextafter(math.ldexp(2688.0, e), 0.0)) == e
