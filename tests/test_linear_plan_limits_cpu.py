"""The plan's query at the ends of what it may be asked: numbers of SMs that hold no pair are refused, any other
gives a plan."""
import ctypes
import os

import pytest

import speculative_decoding_verification_59_gb300 as sv


@pytest.fixture(scope="module", autouse=True)
def lib():
    if not os.path.exists(sv.lib_path()):
        import __graft_entry__
        __graft_entry__.build()
    return sv.load_library()


def test_a_device_without_a_pair_is_refused():
    clusters, plan = (ctypes.c_int32 * 3)(1, 1, 1), (ctypes.c_int32 * 5)()
    for M in (1, 65, 500):
        assert sv.load_library().spec_matmul_plan(M, 64, 128, 1, clusters, plan) == sv.SPEC_ERR_INVALID_ARG


@pytest.mark.parametrize("sms", [2, 3, 7, 160, 161, 1000, 2147483647])
@pytest.mark.parametrize("clusters", [(0, 0, 0), (-1, -5, -2147483648), (2147483647,) * 3])
@pytest.mark.parametrize("sizes", [(65, 1, 1), (65, 64, 2147483391), (2147483391, 1, 128), (70, 2147483391, 1), (5000, 4000, 4096)])
def test_any_other_number_gives_a_plan(sms, clusters, sizes):
    way, W, together, groups, parts = sv.matmul_plan(*sizes, sms, clusters)
    assert way in (sv.SPEC_MATMUL_WHOLE, sv.SPEC_MATMUL_CLUSTERS, sv.SPEC_MATMUL_SHARES)
    assert W in (64, 128, 192, 256) and together in (1, 2) and groups >= 1 and parts >= 1
    assert way != sv.SPEC_MATMUL_SHARES or groups <= 80                                  # what the workspace has room for
