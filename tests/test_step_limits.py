"""Ends of the documented ranges of the drafted step's calls, without a GPU: a call whose arguments
are right stops at the device check."""
import ctypes
import math

import pytest
import torch

import mla_paged_latent_page_amd as mp
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


def test_page_calls_refuse_counts_past_2_30(lib):  # noqa: F811
    d = ctypes.byref(cache_desc())
    for n, status in ((2 ** 30, DEV), (2 ** 30 + 1, SHAPE), (2 ** 31 - 1, SHAPE)):
        assert lib.mla_copy_pages(FAKE, FAKE, n, d, None, None) == status
        assert lib.mla_fork_paged(FAKE, FAKE, FAKE, n, FAKE, d, None, None) == status
        assert lib.mla_compact_paged(FAKE, FAKE, n, d, None, None) == status


@pytest.mark.parametrize("kw", [dict(first_position=2 ** 32), dict(first_position=2 ** 31),
                                dict(original_max_position=2 ** 32 + 4096, scaling="by_parts")])
def test_binding_refuses_positions_that_an_int32_would_cut_off(kw):
    with pytest.raises(ValueError, match=next(iter(kw))):
        mp.mla_rope_freqs(torch.zeros((4, 64)), **kw)
