"""Figures of bench.py's line, on the CPU."""
import bench


def test_small_fractions_stay_positive():
    """A 64x512x512 step with one slow stage among four: 0.05 of 1890 TFLOP/s."""
    assert bench.four_digits(0.05 / 1890) > 0
    assert bench.four_digits(0.5512345) == 0.5512 and bench.four_digits(0.0) == 0.0
