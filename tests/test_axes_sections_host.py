"""Sections of bgg_rotary_axes that are not whole numbers are refused, not cut
to some."""
import numpy as np
import pytest

import bit_gemv_gemm_amd as bgg


@pytest.mark.parametrize("sections", [[16.5, 8], [15.999999, 1], [float("nan"), 8], [float("inf")], ["3"], [1 + 0j], 3, [[3, 2]],
                                      np.float32(4), [2.0 ** 70], np.array([2 ** 64 - 1], np.uint64)])
def test_refused(sections):
    with pytest.raises(ValueError):
        bgg.bgg_rotary_axes(sections)


@pytest.mark.parametrize("sections", [[2, 1], (2, 1), np.array([2, 1], np.int32), np.array([2, 1], np.uint8), [2.0, 1.0],
                                      np.array([2, 9, 1, 9])[::2]])
def test_whole_numbers_of_any_type(sections):
    assert bgg.bgg_rotary_axes(sections).tolist() == [0, 0, 1]
