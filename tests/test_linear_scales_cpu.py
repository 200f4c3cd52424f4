"""Where scales lie and how far apart, as the dense side's calls accept it: what would store two blocks' scales in one
place is refused before the device is touched.  (The calls that pass these checks have no GPU to run on
here, so they are made with rows of no alignment, which is refused after them.)"""
import os

import pytest

import speculative_decoding_verification_59_gb300 as sv
from test_linear_cpu import ALIGN, E4M3, FAKE, INVALID, act, norm, quantize


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(sv.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return sv.load_library()


# the stride between a block's scales and the next one's: at least the rows, or 0 for a single block
ROWS = [(0, 1, 256, INVALID), (0, 3, 256, INVALID), (0, 3, 144, INVALID), (1, 3, 256, INVALID), (1, 3, 128, INVALID), (-4, 1, 256, INVALID),
        (0, 1, 128, ALIGN), (0, 3, 128, ALIGN), (0, 3, 16, ALIGN), (1, 1, 256, ALIGN), (3, 3, 256, ALIGN)]


@pytest.mark.parametrize("pitch,rows,dim,want", ROWS)
def test_scales_of_rows_that_overlap(pitch, rows, dim, want):
    off = FAKE + 2                                           # not aligned: the last check of a call
    assert norm(x=off, ot=E4M3, scale=FAKE, pitch=pitch, rows=rows, dim=dim) == want
    assert act(gate=off, ot=E4M3, scale=FAKE, pitch=pitch, rows=rows, dim=dim) == want
    assert quantize(x=off, pitch=pitch, rows=rows, dim=dim) == want


# a weight's: at least a row's blocks, or 0 for a single row of them
@pytest.mark.parametrize("pitch,rows,dim,want", [
    (0, 129, 128, INVALID), (0, 256, 512, INVALID), (3, 129, 512, INVALID), (3, 128, 512, INVALID), (-1, 129, 128, INVALID), (0, 128, 512, ALIGN),
    (0, 1, 16, ALIGN), (4, 129, 512, ALIGN), (1, 129, 128, ALIGN)])
def test_scales_of_a_weight_that_overlap(pitch, rows, dim, want):
    assert quantize(x=FAKE + 2, high=128, pitch=pitch, rows=rows, dim=dim) == want
