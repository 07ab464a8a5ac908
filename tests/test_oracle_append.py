"""The 64-bit definitions of the rotary append and the 8-bit cache, pinned by hand-worked values (CPU)."""
import numpy as np
import pytest

from oracle import append as A


def test_e4m3_bytes_round_trip_and_border_values():
    for b in range(256):
        if b & 127 != 127:
            assert A.to_byte(A.VALUES[b]) == b
    assert A.VALUES[0x7E] == 448.0 and A.VALUES[0x01] == 2.0 ** -9 and A.VALUES[0x38] == 1.0
    assert A.to_byte(464.0) == 0x7E and A.to_byte(1e9) == 0x7E and A.to_byte(-1e9) == 0xFE    # saturates
    assert A.to_byte(1.0625) == 0x38 and A.to_byte(1.1875) == 0x3A                            # ties to even
    assert A.to_byte(2.0 ** -10) == 0 and A.to_byte(1.5 * 2.0 ** -9) == 2                     # subnormal ties
    assert A.to_byte(np.inf) == 0x7F and A.to_byte(np.nan) == 0x7F
    assert A.to_byte(15.9) == A.to_byte(16.0)                                                 # carries into the exponent


def test_to_byte_is_the_nearest():
    rng = np.random.default_rng(0)
    fin = A.VALUES[np.isfinite(A.VALUES)]
    for y in np.concatenate([rng.normal(size=300), 300 * rng.normal(size=100), 0.01 * rng.normal(size=100)]):
        best = np.abs(fin - np.clip(y, -448, 448)).min()
        assert abs(A.VALUES[A.to_byte(y)] - np.clip(y, -448, 448)) == best
        assert best <= A.half_step(y)


def test_need_is_the_smallest_exponent():
    for a, x in [(448.0, 0), (448.0001, 1), (1.0, -8), (1.75, -8), (1.7501, -7), (0.0, -117), (3e38, 119)]:
        assert A.need(a) == x
    for a in (3.5, 100.0, 7e-5):
        assert a <= 448 * 2.0 ** A.need(a) and a > 448 * 2.0 ** (A.need(a) - 1)


@pytest.mark.parametrize("interleaved", [False, True])
def test_rotation_by_a_quarter_turn(interleaved):
    x = np.arange(1.0, 7.0)[None, None]                      # 6 columns, 4 of them rotated
    table = np.zeros((1, 4))
    table[0, 2:] = 1.0                                       # cos 0, sin 1: (a, b) -> (-b, a)
    want = [-2, 1, -4, 3, 5, 6] if interleaved else [-3, -4, 1, 2, 5, 6]
    assert A.rotate(x, [0], table, interleaved)[0, 0].tolist() == want
    assert A.rotate(x, [-1], table, interleaved)[0, 0].tolist() == x[0, 0].tolist()


def test_append_starts_over_grows_and_keeps():
    cache = np.full((1, 1, 16, 2), 0x7F, np.uint8)
    scale = np.full((1, 1, 1), 255, np.uint8)
    A.append_q8(np.array([[[1.0, -0.5]]]), [0], cache, scale)           # first place: need(1) = -8
    assert scale[0, 0, 0] == 119 and A.values(cache, scale)[0, 0, 0].tolist() == [1.0, -0.5]
    A.append_q8(np.array([[[0.25, 0.0]]]), [1], cache, scale)           # smaller: the scale stays
    assert scale[0, 0, 0] == 119
    A.append_q8(np.array([[[448.0, 1.0]]]), [3], cache, scale)          # larger: all bytes move to 2^0
    assert scale[0, 0, 0] == 127
    assert A.values(cache, scale)[0, 0, [0, 1, 3]].tolist() == [[1.0, -0.5], [0.25, 0.0], [448.0, 1.0]]
    A.append_q8(np.array([[[2.0 ** -8, 1.0]]]), [4], cache, scale)      # under the coarse scale: 2^-8 is two steps
    assert A.values(cache, scale)[0, 0, 4].tolist() == [2.0 ** -8, 1.0]
    A.append_q8(np.array([[[0.25, 0.5]], [[0.1, 0.0]]]), [0, 1], cache, scale)   # the first place again: starts over
    assert scale[0, 0, 0] == 127 + A.need(0.5)
