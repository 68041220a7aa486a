"""The MXFP4 helper of the tests against hand values of the format."""
import numpy as np

import mx_ref


def block(*head):
    v = np.zeros(32)
    v[:len(head)] = head
    return v


def test_ties_go_to_the_even_code_and_large_values_saturate():
    # scale 1: the largest magnitude 4..7.99 has floor(log2) = 2
    code, s = mx_ref.quantise(block(6.0, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 7.9, -0.2))
    assert s[0] == 127
    assert code[:10].tolist() == [7, 0, 2, 2, 4, 4, 6, 6, 7, 8]


def test_scales_follow_the_largest_magnitude():
    for m, byte in ((1.0, 125), (0.999, 124), (2.0 ** -126, 0), (2.0 ** -149, 0), (2.0 ** 127, 252), (0.0, 127)):
        assert mx_ref.quantise(block(m))[1][0] == byte, m
    code, s = mx_ref.quantise(block(1.0, np.inf))
    assert s[0] == 255 and not code.any()
    assert np.isnan(mx_ref.values(mx_ref.pack(code), s)).all()


def test_values_of_codes():
    code = np.arange(32) % 16
    v = mx_ref.values(mx_ref.pack(code.astype(np.uint8)), np.array([128], dtype=np.uint8))
    want = np.concatenate((mx_ref.GRID, -mx_ref.GRID)) * 2
    assert np.array_equal(v, np.tile(want, 2))
    assert np.array_equal(mx_ref.unpack(mx_ref.pack(code)), code)
