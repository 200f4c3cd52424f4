"""How a product's row scales have to lie, before the device is touched: a single row's, and those of more than 64
rows, anywhere; of 2 to 64 rows at 16 bytes, blocks a multiple of 4 apart.  (What passes is refused after it, for its
workspace: no kernel is launched here.)"""
import os

import pytest

import speculative_decoding_verification_59_gb300 as sv
from test_linear_cpu import ALIGN, FAKE, INVALID, matmul

SMALL = sv.SPEC_ERR_WORKSPACE_TOO_SMALL


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(sv.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return sv.load_library()


@pytest.mark.parametrize("M,at,stride,want", [
    (1, 4, 4, SMALL), (1, 0, 1, SMALL), (1, 12, 7, SMALL), (65, 4, 65, SMALL), (65, 8, 68, SMALL), (300, 0, 301, SMALL),
    (2, 4, 4, ALIGN), (64, 8, 64, ALIGN), (2, 0, 2, ALIGN), (64, 0, 65, ALIGN), (64, 0, 64, SMALL),
    (1, 2, 4, ALIGN), (65, 2, 68, ALIGN), (64, 2, 64, ALIGN),
    (1, 0, 0, INVALID), (65, 0, 64, INVALID), (1, 0, 1 << 38, INVALID)])
def test_row_scales(M, at, stride, want):
    assert matmul(M=M, xs=FAKE + at, xss=stride, wb=16) == want
    if want != INVALID and stride != 7 and stride % 4:       # of one block the stride is not used
        assert matmul(M=M, xs=FAKE + at, xss=stride, wb=16, K=128) == SMALL
