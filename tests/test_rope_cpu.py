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


def test_in_place_with_other_strides_is_refused(sdv):  # noqa: F811
    """A row that is written where another one is still to be read."""
    r, p = rope(sdv), pages(sdv)
    assert rows(sdv, r, xs=1024, os=1028) == EINVAL and rows(sdv, r, xs=2048, os=1024) == EINVAL
    assert append(sdv, p, r, o_sm=1028, o_sb=5 * 1028) == EINVAL
    assert append(sdv, p, r, o_sb=6 * 1024) == EINVAL
    assert append(sdv, p, r, B=1, o_sm=2048) == EINVAL
