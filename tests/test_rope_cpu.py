"""Rotary calls: sizes and places that are refused before anything is launched (no GPU needed)."""
import pytest

from test_samples_cpu import A, EINVAL, EUNSUPPORTED, append, pages, rope, rows, sdv  # noqa: F401


@pytest.mark.parametrize("heads", [2 ** 31 - 1, 2 ** 31 - 100, 2 ** 31 - 511, 2 ** 30])
def test_more_heads_than_a_grid_has_places_are_refused(sdv, heads):  # noqa: F811
    for D in (8, 64, 128, 1024):
        assert rows(sdv, rope(sdv, rot=8), N=1, heads=heads, D=D) == EUNSUPPORTED
    for D in (64, 128, 256):
        p = pages(sdv, D=D, row_stride=D, head_stride=16 * D, page_stride=4 * 16 * D)
        assert append(sdv, p, rope(sdv, rot=8), B=1, M=1, H=heads) == EUNSUPPORTED
