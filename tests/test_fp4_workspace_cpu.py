"""A decode workspace sized for a batch serves every smaller one (host only)."""
import fp4_workspace as F


def test_smaller_batches():
    F.check_smaller_batches()


def test_shorter_bounds_and_windows():
    F.check_shorter_bounds_and_windows()


def test_not_wasteful():
    F.check_not_wasteful()


def test_given_ranges():
    F.check_given_ranges()
