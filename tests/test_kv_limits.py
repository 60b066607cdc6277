"""Limits of the cache and answer calls that the host alone decides: no GPU needed."""

import pytest

import verify_draft_prep_gb300 as sd


@pytest.fixture(scope="module")
def lib():
    sd.build()
    return sd.load()


@pytest.mark.parametrize("D", [16, 64, 80, 128])
def test_attend_scratch_has_room_to_be_aligned(lib, D):
    """The parts are written 32 bytes at a time and take a whole number of them; a caller's scratch
    begins at any multiple of 16, so there are 16 bytes more than the parts take."""
    assert lib.sd_kv_attend_workspace_bytes(D) % 32 == 16
