"""Ends of the documented ranges of the drafted step's calls, without a GPU: a call whose arguments
are right stops at the device check."""
import ctypes
import math

from test_step_host import DEV, FAKE, SHAPE, cache_desc, freqs, lib  # noqa: F401


def test_rope_freqs_reach_is_that_of_the_last_row(lib):  # noqa: F811
    # position 0 has no angle, whatever the frequency
    assert freqs(lib, rows=1, scaling=1, factor=1e-300) == DEV
    assert freqs(lib, rows=2, scaling=1, factor=1e-300) == SHAPE
    # the largest frequency is 1 / factor: 2^50 quarter turns at position 1000
    factor = 1000 / (2.0 ** 50 * math.pi / 2)
    assert freqs(lib, first=993, rows=7, scaling=1, factor=factor) == DEV      # up to position 999
    assert freqs(lib, first=993, rows=9, scaling=1, factor=factor) == SHAPE    # up to 1001


def test_free_refuses_pools_whose_counts_its_walk_cannot_number(lib):  # noqa: F811
    def free(pages):
        return lib.mla_free_paged(FAKE, 3, FAKE, FAKE, FAKE, ctypes.byref(cache_desc(pages=pages)), None)
    assert free(2 ** 31 - 1) == DEV and free(2 ** 31) == SHAPE and free(2 ** 32 - 1) == SHAPE
