"""Pins of the MXFP4 definition the GPU tests compare with (no GPU)."""
import numpy as np

import _mxfp4_reference as mx


def test_every_code_decodes_to_its_value():
    packed = np.array([[c | (c << 4) for c in range(16)]], dtype=np.uint8)
    v = mx.decode(packed, np.array([[127]], dtype=np.uint8), 32)[0]
    want = [0, .5, 1, 1.5, 2, 3, 4, 6, 0, -.5, -1, -1.5, -2, -3, -4, -6]
    assert np.array_equal(v, np.repeat(want, 2)) and np.signbit(v[16])


def test_values_of_the_format_come_back():
    rng = np.random.default_rng(1)
    code = rng.integers(0, 16, (40, 3, 32)).astype(np.uint8)
    code[..., 0] = 7                                  # a 6 in each block fixes its scale
    s = rng.integers(1, 250, (40, 3)).astype(np.uint8)
    v = mx.decode(mx.pack(code), s, 96)
    back, s2 = mx.encode(v)
    assert np.array_equal(s2, s) and np.array_equal(back, code)


def test_ties_go_to_the_even_code_and_scales_to_the_smallest():
    mid = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, -0.25, -0.75, -2.5, -5.0, 6.0]
    code, s = mx.encode(np.array([mid + [0.0] * 20]))
    assert s[0, 0] == 127
    assert code[0, 0, :12].tolist() == [0, 2, 2, 4, 4, 6, 6, 8, 10, 12, 14, 7]
    for amax, X in ((6.0, 0), (6.0001, 1), (3.0, -1), (0.0, -127), (6 * 2.0 ** -127, -127), (7 * 2.0 ** -127, -126),
                    (2.0 ** -149, -127), (3.4e38, 126)):
        assert mx.encode(np.array([[amax]]))[1][0, 0] == X + 127


def test_blocks_that_are_not_finite():
    v = np.ones((1, 96))
    v[0, 40], v[0, 70] = np.nan, -np.inf
    code, s = mx.encode(v)
    assert s[0].tolist() == [125, 255, 255] and not code[0, 1:].any()
    d = mx.decode(mx.pack(code), s, 96)[0]
    assert np.array_equal(d[:32], np.ones(32)) and np.isnan(d[32:]).all()
