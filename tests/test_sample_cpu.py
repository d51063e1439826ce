"""Sampling: places that are refused before anything is launched (no GPU needed)."""
from test_samples_cpu import A, EINVAL, draw, sdv  # noqa: F401


def test_outputs_in_the_settings_place_are_refused(sdv):  # noqa: F811
    """A large batch's rows look at all settings for their place in the order, when earlier rows may be drawn already."""
    assert draw(sdv, k=A, tokens=A) == EINVAL
    assert draw(sdv, T=2 * A, prob=2 * A) == EINVAL
    assert draw(sdv, p=2 * A, prob=2 * A) == EINVAL
